"""The tensor front end of the added calls, as far as it goes without a GPU: what it refuses, and how."""
import os

import pytest
import torch

from gate_cores_b200 import build, cores

X = torch.zeros(4, 64)
ROW = torch.zeros(4, 2, dtype=torch.int32)


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_it_is_built_and_loaded():
    assert os.path.exists(build.FRONT)
    assert cores._front.__file__ == build.FRONT


@pytest.mark.parametrize("call", [
    lambda: cores.layer_norm(X), lambda: cores.layer_norm_backward(X, X), lambda: cores.rope(X, None, X),
    lambda: cores.rope_backward(X, None, X), lambda: cores.expert_sort(ROW, 4), lambda: cores.expert_dispatch(X, ROW),
    lambda: cores.expert_dispatch_backward(X, ROW), lambda: cores.expert_combine(X, ROW),
    lambda: cores.expert_combine_backward(X, X, ROW),
    lambda: cores._front.layer_norm(X, None, None, 0.0, 1e-6, None),
    lambda: cores._front.layer_norm_backward(X, X, None, 0.0, 1e-6, None, True, True, None),
    lambda: cores._front.rope(X, None, X, None, None, 0, 1.0, None, None, False),
    lambda: cores._front.expert_sort(ROW, 4, None), lambda: cores._front.expert_dispatch(X, ROW, None),
    lambda: cores._front.expert_combine(X, ROW, None, None, False),
    lambda: cores._front.expert_combine_backward(X, X, ROW, None, None, True)])
def test_tensors_of_the_host(call):
    with pytest.raises(ValueError, match="CUDA device"):
        call()


@pytest.mark.parametrize("call,words", [
    (lambda f: f.layer_norm(X), "takes 6 arguments .1 given"),
    (lambda f: f.layer_norm(3, None, None, 0.0, 1e-6, None), "x must be a tensor"),
    (lambda f: f.layer_norm(X, 3, None, 0.0, 1e-6, None), "gain must be a tensor"),
    (lambda f: f.layer_norm(X, None, None, "a", 1e-6, None), "real number"),
    (lambda f: f.expert_sort(ROW, 4.5, None), None),
    (lambda f: f.expert_sort(ROW), "takes 3 arguments"),
    (lambda f: f.rope(X, None, None, None, None, 0, 1.0, None, None, False), "inv_freq must be a tensor")])
def test_arguments_of_other_types(call, words):
    with pytest.raises(TypeError, match=words):
        call(cores._front)
