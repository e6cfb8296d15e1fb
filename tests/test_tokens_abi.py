"""Refusals of the token-side calls on the host (no GPU needed): every bad argument is turned
down before anything is launched."""
import pytest

import block_draft_model_proj_gb300 as dflash
from block_draft_model_proj_gb300 import build as dbuild

BF16, F32, F16 = dflash.DFLASH_DTYPE_BF16, dflash.DFLASH_DTYPE_F32, dflash.DFLASH_DTYPE_F16
P = 4096   # an aligned address that is never read: each call below is refused
BAD, NOT = dflash.DFLASH_ERR_INVALID_ARG, dflash.DFLASH_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def cpu_lib():
    dbuild.build()
    return dflash.load()


def _call(fn, good, **kw):
    args = dict(good)
    args.update(kw)
    return fn(*args.values())


SAMPLE = dict(logits=P, dt=BF16, ld=100, R=4, V=100, t=None, k=None, p=None, m=None, per=2, u=P,
              tok=P, probs=None, ws=None, n=0, stream=None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(R=-1)), (BAD, dict(V=0)), (BAD, dict(ld=99)), (BAD, dict(per=0)),
    (BAD, dict(per=3)), (BAD, dict(dt=F16)), (BAD, dict(dt=7)), (BAD, dict(logits=None)),
    (BAD, dict(u=None)), (BAD, dict(tok=None)), (BAD, dict(logits=P + 1)),
    (BAD, dict(dt=F32, logits=P + 2)), (BAD, dict(probs=P + 2)),
    (NOT, dict(V=(1 << 19) + 1, ld=1 << 20)), (NOT, dict(R=(1 << 24) + 2))])
def test_sample_refusals(cpu_lib, want, kw):
    assert _call(cpu_lib.dflash_sample_tokens, SAMPLE, **kw) == want
    assert cpu_lib.dflash_last_error()


VERIFY = dict(logits=P, dt=BF16, t=None, k=None, p=None, m=None, q=P, draft=P, B=2, gamma=3, V=100,
              u=P, eos=-1, em=P, ne=P, ac=P, ws=P, n=1 << 20, stream=None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(B=0)), (BAD, dict(gamma=-1)), (BAD, dict(V=0)), (BAD, dict(dt=F16)),
    (BAD, dict(logits=None)), (BAD, dict(q=None)), (BAD, dict(draft=None)), (BAD, dict(u=None)),
    (BAD, dict(em=None)), (BAD, dict(ne=None)), (BAD, dict(ac=None)), (BAD, dict(ws=None)),
    (BAD, dict(n=0)), (BAD, dict(ws=P + 16)), (BAD, dict(logits=P + 1)),
    (NOT, dict(V=(1 << 19) + 1)), (NOT, dict(B=1 << 24)), (NOT, dict(B=1 << 30, gamma=1 << 30))])
def test_verify_refusals(cpu_lib, want, kw):
    assert _call(cpu_lib.dflash_verify_sampling_filtered, VERIFY, **kw) == want
    assert cpu_lib.dflash_last_error()


EMBED = dict(table=P, dt=BF16, V=10, D=64, ids=P, T=5, scale=1.0, out=P, stream=None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(V=0)), (BAD, dict(D=0)), (BAD, dict(T=-1)), (BAD, dict(dt=F16)),
    (BAD, dict(table=None)), (BAD, dict(ids=None)), (BAD, dict(out=None)),
    (BAD, dict(table=P + 8)), (BAD, dict(out=P + 2)), (BAD, dict(scale=float("nan"))),
    (BAD, dict(scale=float("inf"))), (NOT, dict(D=(1 << 20) + 1))])
def test_embed_refusals(cpu_lib, want, kw):
    assert _call(cpu_lib.dflash_embed_tokens, EMBED, **kw) == want
    assert cpu_lib.dflash_last_error()


GRAD = dict(g=P, gdt=BF16, ids=P, T=5, V=10, D=64, scale=1.0, acc=0, table=P, tdt=F32, ws=P,
            n=1 << 30, stream=None)


@pytest.mark.parametrize("want,kw", [
    (BAD, dict(V=0)), (BAD, dict(D=0)), (BAD, dict(T=-1)), (BAD, dict(gdt=F16)),
    (BAD, dict(tdt=F16)), (BAD, dict(g=None)), (BAD, dict(ids=None)), (BAD, dict(table=None)),
    (BAD, dict(g=P + 8)), (BAD, dict(table=P + 4)), (BAD, dict(ws=None)), (BAD, dict(n=100)),
    (BAD, dict(ws=P + 16)), (BAD, dict(scale=float("nan"))), (NOT, dict(D=(1 << 20) + 1))])
def test_grad_refusals(cpu_lib, want, kw):
    assert _call(cpu_lib.dflash_embed_tokens_grad, GRAD, **kw) == want
    assert cpu_lib.dflash_last_error()


def test_nothing_to_do(cpu_lib):
    assert _call(cpu_lib.dflash_sample_tokens, SAMPLE, R=0, logits=None, u=None, tok=None) == 0
    assert _call(cpu_lib.dflash_embed_tokens, EMBED, T=0, ids=None, out=None) == 0


def test_binding_refuses_other_tensors(cpu_lib):
    torch = pytest.importorskip("torch")
    x, u, t = torch.zeros((4, 10)), torch.zeros(4), torch.zeros(4, dtype=torch.int32)
    if not torch.cuda.is_available():
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            dflash.dflash_sample_tokens(x, u, t)        # not on a CUDA device
    with pytest.raises(ValueError):
        dflash.dflash_sample_tokens(x.half(), u, t)
    with pytest.raises(ValueError):
        dflash.dflash_sample_tokens(x, u, t, rows_per_request=3)
    with pytest.raises(ValueError):
        dflash.dflash_embed_tokens(x, t.long(), x)
    with pytest.raises(ValueError):
        dflash.dflash_embed_tokens_grad(x.double(), t, x)


@pytest.mark.parametrize("name,good,kws", [
    ("dflash_sample_tokens", SAMPLE, ("t", "k", "p", "m", "u", "tok")),
    ("dflash_verify_sampling_filtered", VERIFY, ("t", "k", "p", "m", "q", "draft", "u", "em", "ne",
                                                 "ac")),
    ("dflash_embed_tokens", EMBED, ("ids",)), ("dflash_embed_tokens_grad", GRAD, ("ids",))])
def test_pointers_off_their_elements(cpu_lib, name, good, kws):
    for kw in kws:
        for off in (1, 2, 3):
            assert _call(getattr(cpu_lib, name), good, **{kw: P + off}) == BAD, (kw, off)
            assert b"aligned" in cpu_lib.dflash_last_error()


@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 200, (1 << 31) - 2048])
def test_gradient_workspace_of_the_most_slots(cpu_lib, T):
    """Two buffers of sorted tokens and of their slots, whatever the rounding up to chunks."""
    n = cpu_lib.dflash_embed_tokens_grad_workspace_size(2, 1, T)
    assert 16 * T <= n <= 32 * T


@pytest.mark.parametrize("dt,ld,probs", [
    (F32, 100, P), (F32, 120, P), (BF16, 100, P), (F32, 100, P + 4), (F32, 100, P + 4 * 399),
    (F32, 120, P + 4 * 459), (F32, 1 << 40, P + 4 * (3 << 40)), (F32, 100, P - 4 * 399),
    (F32, (1 << 62) + 7, P + (1 << 20))])
def test_probabilities_in_the_logits(cpu_lib, dt, ld, probs):
    """[4, 100] rows: probabilities that would be written over logits still to be read."""
    at = 1 << 30
    kw = dict(logits=at, dt=dt, ld=ld, probs=probs - P + at)
    assert _call(cpu_lib.dflash_sample_tokens, SAMPLE, **kw) == BAD
    assert b"overlap" in cpu_lib.dflash_last_error()
