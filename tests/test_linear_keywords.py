"""The allocating forms of the linear layer's operators take every argument by its
documented name, and show their signatures."""
import inspect

import pytest
import torch

import dense_gemm_matrix_amd as dg

FORMS = {"linear": "A B bias act residual out_dtype keep_preact in_fmt",
         "linear_backward": "A B dC preact act bias in_fmt",
         "matmul_f8": "A B scale_a scale_b bias act residual out_dtype",
         "rms_norm": "X weight residual f8 keep eps",
         "rms_norm_backward": "dY total weight rstd dtotal",
         "quantize_f8": "X transpose"}


@pytest.mark.parametrize("name", list(FORMS))
def test_signatures_are_shown(name):
    fn = getattr(dg, name)
    assert list(inspect.signature(fn).parameters) == FORMS[name].split() + ["stream"]
    assert fn.__name__ == name and fn.__doc__


def operands(device):
    t = lambda *s, dtype=torch.float32: torch.ones(*s, device=device).to(dtype)  # noqa: E731
    f8 = dg._linear.F8
    return {"linear": dict(A=t(4, 8), B=t(8, 16), act="silu"),
            "linear_backward": dict(A=t(4, 8), B=t(8, 16), dC=t(4, 16), bias=True),
            "matmul_f8": dict(A=t(4, 16, dtype=f8), B=t(8, 16, dtype=f8), scale_a=t(4), scale_b=t(8)),
            "rms_norm": dict(X=t(4, 8), weight=t(8), keep=True),
            "rms_norm_backward": dict(dY=t(4, 8), total=t(4, 8), weight=t(8), rstd=t(4)),
            "quantize_f8": dict(X=t(4, 8))}


@pytest.mark.parametrize("name", list(FORMS))
def test_keyword_calls_reach_the_operator(name):
    """On the CPU: the refusal of a host tensor, not of the call's form."""
    kw = operands("cpu")[name]
    with pytest.raises(ValueError, match="device tensor"):
        getattr(dg, name)(**kw)
    with pytest.raises(TypeError, match=f"{name}.*missing"):
        getattr(dg, name)()


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(FORMS))
def test_keyword_calls_give_the_same(name):
    kw = operands("cuda")[name]
    fn = getattr(dg, name)
    first = next(iter(kw))
    rest = {k: v for k, v in kw.items() if k != first}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    results = [fn(kw[first], **rest), fn(**kw), fn(**kw, stream=side), fn(**kw, stream=None)]
    torch.cuda.synchronize()
    flat = lambda r: [v for v in (r.values() if isinstance(r, dict) else r if isinstance(r, tuple) else (r,))  # noqa: E731
                      if v is not None]
    for r in results[1:]:
        assert all(torch.equal(a.float(), b.float()) for a, b in zip(flat(r), flat(results[0])))
