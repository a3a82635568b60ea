"""What the learner operators' binding refuses before the library is called:
tensors that no kernel may be given as device memory.  The tensors here are
stand-ins that say of themselves where they are; nothing is launched."""
import pytest

torch = pytest.importorskip("torch")
import nvfp4_w4a4_moe_top_gb300 as M  # noqa: E402

B16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


class Stand:
    """Says it is a contiguous tensor on `device` (-1: the host)."""

    def __init__(self, shape, dtype, device=0, contiguous=True):
        self.shape, self.dtype, self.device, self.flat = torch.Size(shape), dtype, device, contiguous

    is_cuda = property(lambda self: self.device >= 0)

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return self.flat

    def stride(self):
        st, n = [], 1
        for s in reversed(self.shape):
            st.insert(0, n)
            n *= s
        return tuple(st)

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return 1 << 20

    def __getitem__(self, i):
        raise AssertionError("read")


class Library:
    """Counts the calls that reach it and accepts them."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*a):
            self.calls += 1
            return 1 << 40 if name.endswith("_bytes") else 0
        return call


@pytest.fixture
def library(monkeypatch):
    fake = Library()
    monkeypatch.setattr(M, "lib", lambda: fake)
    M._dt()
    monkeypatch.setattr(M._types, "device", lambda: 0)
    monkeypatch.setattr(M._types, "raw_stream", lambda device: 0)
    return fake


T, V, K, D, N = 4, 100, 3, 128, 2


def operators():
    """Name -> (call, its tensors by name)."""
    s = lambda *shape, t=F32: Stand(shape, t)  # noqa: E731
    logits = dict(logits=s(T, V, t=B16))
    teacher = dict(teacher_ids=s(T, K, t=I32), teacher_logits=s(T, K), teacher_lse=s(T))
    row = dict(x=s(T, D, t=B16), res=s(T, D, t=B16), w=s(D, t=B16), h=s(T, D, t=B16), y=s(T, D, t=B16),
               y8=s(T, D, t=U8), y8_sf=s(512, t=U8), rstd=s(T), status=s(1, t=I32))
    back = dict(dy=s(T, D, t=B16), dh=s(T, D, t=B16), h=s(T, D, t=B16), rstd=s(T), w=s(D, t=B16), dx=s(T, D, t=B16),
                dw=s(D), ws=s(4096, t=U8), status=s(1, t=I32))
    lp = dict(logits, targets=s(T, t=I32), logprob=s(T), entropy=s(T), stats=s(T, 2), top_ids=s(T, N, t=I32),
              top_logprob=s(T, N), status=s(1, t=I32))
    lpb = dict(logits, targets=s(T, t=I32), stats=s(T, 2), entropy=s(T), g_logprob=s(T), g_entropy=s(T),
               dlogits=s(T, V, t=B16), status=s(1, t=I32))
    ds = dict(logits, **teacher, loss=s(T), stats=s(T, 4), status=s(1, t=I32))
    dsb = dict(logits, **teacher, stats=s(T, 4), g=s(T), dlogits=s(T, V, t=B16), status=s(1, t=I32))
    dst = dict(logits, **teacher, g=s(T), loss=s(T), dlogits=s(T, V, t=B16), status=s(1, t=I32))
    return {
        "norm": (lambda **a: M.moe_add_rmsnorm(eps=1e-6, **a), row),
        "norm gradient": (lambda **a: M.moe_add_rmsnorm_backward(**a), back),
        "log-probabilities": (lambda **a: M.moe_token_logprobs(inv_temperature=1.0, n_top=N, **a), lp),
        "their gradient": (lambda **a: M.moe_token_logprobs_backward(inv_temperature=1.0, **a), lpb),
        "distillation": (lambda **a: M.moe_distill_topk(inv_temperature=1.0, **a), ds),
        "its gradient": (lambda **a: M.moe_distill_topk_backward(inv_temperature=1.0, **a), dsb),
        "its step": (lambda **a: M.moe_distill_topk_train(inv_temperature=1.0, **a), dst),
    }


@pytest.mark.parametrize("name", list(operators()))
def test_tensors_off_the_current_device(library, name):
    """Every tensor argument, one at a time on the host and on another device."""
    call, args = operators()[name]
    call(**args)
    assert library.calls >= 1
    for what, t in args.items():
        for device in [-1, 1]:
            bad = Stand(t.shape, t.dtype, device)
            library.calls = 0
            with pytest.raises(ValueError):
                call(**{**args, what: bad})
            assert library.calls == 0 or what == "y8_sf", (what, device)
    every = {k: Stand(t.shape, t.dtype, 1) for k, t in args.items()}
    with pytest.raises(ValueError):  # all on a device that is not the current one
        call(**every)


@pytest.mark.parametrize("name", list(operators()))
def test_status_words_of_other_kinds(library, name):
    call, args = operators()[name]
    for bad in [Stand((1,), torch.int64), Stand((1,), F32), Stand((4,), U8), Stand((0,), I32)]:
        library.calls = 0
        with pytest.raises(ValueError):
            call(**{**args, "status": bad})
        assert library.calls == 0
    call(**{**args, "status": None})
    call(**{**args, "status": Stand((8,), I32)})


def test_workspaces(library):
    call, args = operators()["norm gradient"]
    with pytest.raises(ValueError):
        call(**{**args, "ws": Stand((64, 64), U8, contiguous=False)})
    call(**{**args, "ws": Stand((1024,), F32)})
    call(**{**args, "ws": None, "dw": None})


def test_sizes_beyond_32_bits(library):
    """Rows that the library's int cannot count are refused, not counted modulo
    2^32."""
    big = (1 << 32) + 4
    for shape in [(big, 1), (1, big), (1 << 31, 1)]:
        with pytest.raises(ValueError):
            M.moe_token_logprobs(Stand(shape, B16), None, 1.0, 0, None, None, Stand((shape[0], 2), F32))
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm(Stand((big, D), B16), None, Stand((D,), B16), 1e-6, None, Stand((big, D), B16))
    x = Stand((big, D), B16)
    with pytest.raises(ValueError):
        M.moe_add_rmsnorm_backward(x, None, x, Stand((big,), F32), Stand((D,), B16), x, None, None)
    with pytest.raises(ValueError):
        M.moe_distill_topk(Stand((T, V), B16), Stand((T, big), I32), Stand((T, big), F32), None, 1.0, Stand((T,), F32), None)
    assert library.calls == 0
