"""What the embedding and loss entry points refuse, on the host before any
CUDA call, and their workspace sizes.  The addresses are made up, so these
run only where no GPU could be handed them."""
import ctypes

import numpy as np
import pytest

import newton_schulz_fp32_gb300 as nsg


def _gpu():
    try:
        import torch
    except ImportError:
        return False
    return torch.cuda.is_available()


pytestmark = pytest.mark.skipif(_gpu(), reason="made-up addresses stay away from a GPU")

FAKE = 1 << 20   # a non-NULL, aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    nsg.build()
    return nsg.lib()


def refused(lib, rc, word, code=nsg.MUON_ERR_INVALID):
    assert rc == code, (rc, lib.muon_last_error())
    assert word in lib.muon_last_error().decode(), (word, lib.muon_last_error())


LOOKUP = dict(table=FAKE, tt=0, ts=64, rows=10, cols=64, ids=FAKE, it=1, n=4, scale=1.0,
              out=FAKE + (1 << 16), ot=0, os=64, stream=None)


@pytest.mark.parametrize("change,word", [
    (dict(table=None), "table is NULL"), (dict(table=FAKE + 1), "table is NULL or misaligned"),
    (dict(ids=None), "NULL"), (dict(out=None), "NULL"), (dict(ids=FAKE + 4), "aligned"),
    (dict(out=FAKE + (1 << 16) + 1), "aligned"), (dict(tt=2), "table_dtype"), (dict(ot=-1), "out_dtype"),
    (dict(it=2), "ids_type"), (dict(rows=0), "rows or cols"), (dict(cols=0), "rows or cols"),
    (dict(n=-1), "n_tokens"), (dict(n=(1 << 30) + 1), "n_tokens"), (dict(ts=63), "table_stride"),
    (dict(os=63), "out_stride"), (dict(scale=float("nan")), "scale"), (dict(scale=float("inf")), "scale"),
    (dict(out=FAKE + 64), "overlaps")])
def test_lookup_refuses(lib, change, word):
    refused(lib, lib.muon_embedding(*dict(LOOKUP, **change).values()), word)


def grad_args(param=(0, 10, 64, 0, 0), parts=None, **change):
    p = np.array([param], dtype=nsg.PARAM_DTYPE)
    q = np.array(parts or [], dtype=nsg.PART_DTYPE)
    a = dict(accum=FAKE, ae=1 << 20, dout=FAKE, dt=0, ds=64, ids=FAKE, it=1, n=4096, scale=1.0, overwrite=0,
             pp=p.ctypes.data, qq=q.ctypes.data if len(q) else None, nparts=len(q), ws=FAKE,
             wb=1 << 24, stream=None)
    a.update(change)
    return list(a.values()), (p, q)


@pytest.mark.parametrize("change,word", [
    (dict(accum=None), "accum"), (dict(accum=FAKE + 4), "accum"), (dict(dout=None), "NULL"),
    (dict(dt=5), "dout_dtype"), (dict(ds=63), "dout_stride"), (dict(it=-1), "ids_type"), (dict(n=-1), "n_tokens"),
    (dict(scale=float("nan")), "scale"), (dict(overwrite=2), "overwrite"), (dict(ws=None), "workspace"),
    (dict(ws=FAKE + 8), "workspace"), (dict(wb=100), "workspace"), (dict(pp=None), "param"),
    (dict(ae=639), "accum_elems"), (dict(ae=-1), "accum_elems"), (dict(nparts=1), "parts is NULL"), (dict(nparts=-1), "parts is NULL")])
def test_gradient_refuses(lib, change, word):
    args, _keep = grad_args(**change)
    refused(lib, lib.muon_embedding_grad(*args), word)


@pytest.mark.parametrize("param,parts,word,code", [
    ((-1, 10, 64, 0, 0), None, "offset", -1), ((0, 0, 64, 0, 0), None, "rows or cols", -1),
    ((0, 10, 64, 0, 0), [(0, 600, 0)], "covered", -1),
    ((0, 10, 64, 0, 0), [(0, 300, 0), (320, 700, 400)], "covered", -1),
    ((0, 10, 64, 0, 0), [(300, 700, 300), (0, 300, 0)], "sorted", -1),
    ((0, 10, 64, 0, 0), [(0, 300, 0), (300, 700, 200)], "storage", -1),
    ((0, 10, 64, 0, 0), [(0, 700, -4)], "bad range", -1),
    ((0, 10, 64, 0, 0), [(0, 320, 0), (320, 700, (1 << 20) - 300)], "accum_elems", -1),
    ((0, 10, 64, 0, 0), [(4 * i, 4 * i + 4, 4 * i) for i in range(160)], "MAX_SEGMENTS", -2)])
def test_gradient_refuses_tables(lib, param, parts, word, code):
    args, _keep = grad_args(param, parts)
    refused(lib, lib.muon_embedding_grad(*args), word, code)


ROWS = dict(logits=FAKE, dtype=0, stride=100, n=4, vocab=100, targets=FAKE, tt=1)
BAD_ROWS = [
    (dict(logits=None), "NULL"), (dict(logits=FAKE + 1), "aligned"), (dict(dtype=2), "dtype"),
    (dict(stride=99), "stride"), (dict(n=-1), "n_tokens"), (dict(n=1 << 31), "n_tokens"), (dict(vocab=0), "vocab"),
    (dict(targets=None), "NULL"), (dict(targets=FAKE + 4), "aligned"), (dict(tt=3), "targets_type"),
    (dict(scale=0.0), "logit_scale"), (dict(scale=-1.0), "logit_scale"), (dict(scale=float("inf")), "logit_scale"),
    (dict(logp=None), "NULL"), (dict(logp=FAKE + 2), "aligned")]
BAD_GRAD = [
    (dict(d=FAKE + (1 << 16) + 1), "dlogits"), (dict(ds=99), "dlogits_stride"), (dict(d=FAKE, ds=101), "overlaps"),
    (dict(d=FAKE + 2), "overlaps"), (dict(stats=None), "stats"), (dict(stats=FAKE + 2), "stats")]


@pytest.mark.parametrize("change,word", BAD_ROWS)
def test_logprobs_refuse(lib, change, word):
    a = dict(ROWS, scale=1.0, logp=FAKE, stream=None)
    a.update(change)
    refused(lib, lib.muon_token_logprobs(*a.values()), word)


@pytest.mark.parametrize("change,word", BAD_ROWS + BAD_GRAD + [
    (dict(adv=None), "advantages"), (dict(w=None), "weights"), (dict(old=FAKE + 1), "aligned"),
    (dict(lo=-0.1), "clip_low"), (dict(hi=float("nan")), "clip_high"), (dict(kl=float("inf")), "kl_coef"),
    (dict(kl=-0.1), "kl_coef"), (dict(kl=0.1, ref=None), "ref_logp")])
def test_policy_loss_refuses(lib, change, word):
    a = dict(ROWS, adv=FAKE, w=FAKE, old=FAKE, ref=FAKE, lo=0.2, hi=0.2, kl=0.0, scale=1.0, stats=FAKE,
             logp=FAKE, d=FAKE + (1 << 16), ds=100, stream=None)
    a.update(change)
    refused(lib, lib.muon_policy_loss(*a.values()), word)


@pytest.mark.parametrize("change,word", BAD_ROWS + BAD_GRAD + [
    (dict(offsets=None), "offsets"), (dict(ot=2), "offsets_type"), (dict(offsets=FAKE + 4), "misaligned"),
    (dict(pairs=-1), "n_pairs"), (dict(margins=None), "margins"), (dict(beta=float("nan")), "beta"),
    (dict(ls=-0.1), "label_smoothing"), (dict(ls=1.1), "label_smoothing"), (dict(ls=float("nan")), "label_smoothing"),
    (dict(ws=None), "workspace"), (dict(ws=FAKE + 8), "workspace"), (dict(wb=16), "workspace")])
def test_preference_loss_refuses(lib, change, word):
    a = dict(ROWS, offsets=FAKE, ot=1, pairs=2, ref=FAKE, pw=None, beta=0.1, ls=0.0, scale=1.0, stats=FAKE,
             margins=FAKE, logp=FAKE, d=FAKE + (1 << 16), ds=100, ws=FAKE, wb=1 << 20, stream=None)
    a.update(change)
    refused(lib, lib.muon_preference_loss(*a.values()), word)


def test_workspace_sizes(lib):
    assert nsg.embedding_grad_workspace(0, 8) == 0 and nsg.preference_loss_workspace(0) == 0
    small, large = nsg.embedding_grad_workspace(2000, 64), nsg.embedding_grad_workspace(20000, 64)
    assert 0 < small < large
    assert nsg.preference_loss_workspace(1000) >= 1000 * 12
    for bad in ((-1, 8), (1 << 31, 8), (10, 0)):
        with pytest.raises(nsg.MuonError):
            nsg.embedding_grad_workspace(*bad)
    with pytest.raises(nsg.MuonError):
        nsg.preference_loss_workspace(-1)
    b = ctypes.c_size_t()
    assert lib.muon_preference_loss_workspace(5, None) == nsg.MUON_ERR_INVALID
    assert lib.muon_preference_loss_workspace(5, ctypes.byref(b)) == nsg.MUON_OK


def test_python_binding_refuses(lib):
    """Wrong types, shapes and devices, before the library is called."""
    import torch
    table, ids = torch.zeros(10, 8), torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA"):
        nsg.embedding(table, ids)
    with pytest.raises(ValueError, match="int32 or int64"):
        nsg.embedding(table, ids.float())
    with pytest.raises(ValueError, match="rows must be contiguous"):
        nsg.embedding(table.t(), ids)
    with pytest.raises(ValueError, match="tokens x cols"):
        nsg.embedding_grad(torch.zeros(80), torch.zeros(2, 8), ids, (0, 10, 8))
    with pytest.raises(ValueError, match="80"):
        nsg.embedding_grad(torch.zeros(79), torch.zeros(3, 8), ids, (0, 10, 8))
    with pytest.raises(ValueError, match="float32"):
        nsg.embedding_grad(torch.zeros(80, dtype=torch.float64), torch.zeros(3, 8), ids, (0, 10, 8))
    z = torch.zeros(3, 8)
    with pytest.raises(ValueError, match="one target per row"):
        nsg.token_logprobs(z, ids[:2])
    with pytest.raises(ValueError, match="CUDA"):
        nsg.policy_loss(z, ids, torch.zeros(3), torch.zeros(3))
    with pytest.raises(ValueError, match="2 \\* pairs"):
        nsg.preference_loss(z, ids, torch.zeros(4, dtype=torch.int64))
