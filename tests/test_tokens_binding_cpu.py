"""What the binding of the operators at the token ends refuses before the
library is called: tensors that no kernel may be given as device memory.  The
tensors are stand-ins that say of themselves where they are."""
import pytest

torch = pytest.importorskip("torch")
import nvfp4_w4a4_moe_top_gb300 as M  # noqa: E402
from test_learner_binding_cpu import Stand, library  # noqa: E402,F401

B16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
T, V, D = 4, 100, 128


def operators():
    """Name -> (call, its tensors by name)."""
    s = lambda *shape, t=F32: Stand(shape, t)  # noqa: E731
    status = dict(status=s(1, t=I32))
    return {
        "embedding": (lambda **a: M.moe_embed_tokens(scale=1.0, **a),
                      dict(ids=s(T, t=I32), table=s(V, D, t=B16), out=s(T, D, t=B16), **status)),
        "its gradient": (lambda **a: M.moe_embed_tokens_backward(scale=1.0, **a),
                         dict(dy=s(T, D, t=B16), ids=s(T, t=I32), dtable=s(V, D), ws=s(1 << 16, t=U8), **status)),
        "draw": (lambda **a: M.moe_sample_tokens(**a),
                 dict(logits=s(T, V, t=B16), u=s(T), tokens=s(T, t=I32), inv_temperature=s(T), top_k=s(T, t=I32),
                      top_p=s(T), min_p=s(T), logprob=s(T), kept_logprob=s(T), **status)),
    }


@pytest.mark.parametrize("name", list(operators()))
def test_tensors_off_the_current_device(library, name):  # noqa: F811
    """Every tensor argument, one at a time on the host and on another device."""
    call, args = operators()[name]
    call(**args)
    assert library.calls == 1
    for what, t in args.items():
        for device in [-1, 1]:
            library.calls = 0
            with pytest.raises(ValueError):
                call(**{**args, what: Stand(t.shape, t.dtype, device)})
            assert library.calls == 0, (what, device)
    with pytest.raises(ValueError):  # all on a device that is not the current one
        call(**{k: Stand(t.shape, t.dtype, 1) for k, t in args.items()})


@pytest.mark.parametrize("name", list(operators()))
def test_types_and_shapes(library, name):  # noqa: F811
    """Every tensor of another type, of another shape, and not contiguous."""
    call, args = operators()[name]
    for what, t in args.items():
        if what == "ws":
            bad = [Stand((64, 64), U8, contiguous=False)]
        elif what == "status":
            bad = [Stand((1,), torch.int64), Stand((0,), I32), Stand((1,), F32)]
        else:
            bad = [Stand(t.shape, torch.float64), Stand(t.shape, torch.int64), Stand(tuple(t.shape) + (2,), t.dtype)]
            if what not in ("logits", "dy", "ids", "dtable", "table"):  # those give the sizes
                bad.append(Stand((t.shape[0] + 1,) + tuple(t.shape[1:]), t.dtype))
            if len(t.shape) == 1 or what == "dtable":
                bad.append(Stand(t.shape, t.dtype, contiguous=False))
        for b in bad:
            library.calls = 0
            with pytest.raises(ValueError):
                call(**{**args, what: b})
            assert library.calls == 0, (what, b.shape, b.dtype)


def test_optional_arguments(library):  # noqa: F811
    call, args = operators()["draw"]
    for what in ["inv_temperature", "top_k", "top_p", "min_p", "logprob", "kept_logprob", "status"]:
        call(**{**args, what: None})
    for what in ["u", "tokens"]:
        with pytest.raises(ValueError):
            call(**{**args, what: None})


def test_sizes_beyond_32_bits(library):  # noqa: F811
    big = (1 << 32) + 4
    with pytest.raises(ValueError):
        M.moe_embed_tokens(Stand((big,), I32), Stand((V, D), B16), 1.0, Stand((big, D), B16))
    with pytest.raises(ValueError):
        M.moe_embed_tokens(Stand((T,), I32), Stand((big, D), B16), 1.0, Stand((T, D), B16))
    with pytest.raises(ValueError):
        M.moe_embed_tokens_backward(Stand((T, D), B16), Stand((T,), I32), 1.0, Stand((big, D), F32), None)
    with pytest.raises(ValueError):
        M.moe_embed_tokens_backward(Stand((big, D), B16), Stand((big,), I32), 1.0, Stand((V, D), F32), None)
    for shape in [(big, 1), (1, big)]:
        with pytest.raises(ValueError):
            M.moe_sample_tokens(Stand(shape, B16), Stand(shape[:1], F32), Stand(shape[:1], I32))
    assert library.calls == 0
