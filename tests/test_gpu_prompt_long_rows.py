"""Every page and every slot of long rows counts: values that name their page or slot.

A value is 1 in one channel and 0 in the others, so that a channel of the output is the sum of the probabilities of a class
of tokens, all positive: test_gpu_prompt.py's bounds are then relative ones (mass = the output itself), 2^-7 for bf16 and
2^-10 for fp16 beside smaller terms, while a lost page takes more than that from its channel (which each case checks on its
oracle).  Three classes one after the other tell apart pages (number mod 128, and number / 128) and slots (mod 128)."""
import numpy as np
import pytest
import torch

from tests import test_gpu_prefix as prefix
from tests import test_gpu_prompt as prompt
from tests.test_gpu_prompt import BF, HF, SCALE, bounds, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


CLASSES = {"page": lambda j, P: j // P % 128, "page / 128": lambda j, P: j // P // 128, "slot": lambda j, P: j % P % 128}


def name_values(vc, table, n, P, of):
    """Value of token j: 1 in channel of(j), but for tokens whose page nothing sees (and the table does not name)."""
    j = torch.arange(n, device="cuda")
    j = j[table[j // P] < vc.shape[0]]
    pages = table[j // P].long()
    vc[pages, :, j % P] = 0.0
    vc[pages, :, j % P, of(j, P)] = 1.0


def oracle(q, kc, parts, P, of, scale, seen):
    """q [n, Hq, 128]; parts: (table row, tokens) one after the other -> the probabilities' sums by class, lse, reach, and
    each whole page's share [n, Hq, pages] and number."""
    hq, hkv = q.shape[1], kc.shape[1]
    j = torch.cat([torch.arange(n, device="cuda") for _, n in parts])
    rows = torch.cat([table[torch.arange(n, device="cuda") // P].long() for table, n in parts])
    k = kc[rows, :, j % P].double()  # [tokens, Hkv, 128]
    out = torch.zeros(q.shape[0], hq, 128, dtype=torch.float64, device="cuda")
    lse, reach = (torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda") for _ in range(2))
    page_of = torch.cat([torch.arange(n, device="cuda") // P + 10 ** 6 * i for i, (_, n) in enumerate(parts)])
    _, page_id = torch.unique(page_of, return_inverse=True)
    whole = torch.bincount(page_id) == P
    shares = torch.zeros(q.shape[0], hq, int(whole.sum()), dtype=torch.float64, device="cuda")
    for h in range(hq):
        x = q[:, h].double()
        s = scale * (x @ k[:, h * hkv // hq].T)
        reach[:, h] = abs(scale) * (x.abs() @ k[:, h * hkv // hq].abs().T).amax(1)
        s = torch.where(seen, s, -torch.inf)
        lse[:, h] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[:, h, None])
        out[:, h].index_add_(1, of(j, P), p)
        per_page = torch.zeros(q.shape[0], len(whole), dtype=torch.float64, device="cuda").index_add_(1, page_id, p)
        shares[:, h] = per_page[:, whole]
    return out, lse, reach, shares, torch.unique(page_of)[whole] % 10 ** 6


def check(got, got_lse, want, lse, reach, count, dt, shares=None, pages=None):
    want, lse, reach, got, got_lse = (np64(t) for t in (want, lse, reach, got, got_lse))
    tol, lse_tol = bounds(want, lse, want, reach, np.full(lse.shape, float(count)), dt)
    if pages is not None:  # a page that were missing would be noticed in every row that sees it
        lost, at = np64(shares), tol[:, :, (pages % 128).cpu().numpy()]
        assert np.all((lost > 2 * at) | (lost == 0))
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], bad.mean(), got[bad][:4], want[bad][:4], tol[bad][:4])
    assert np.all(np.abs(got_lse - lse) <= lse_tol)


@pytest.mark.parametrize("name", list(CLASSES))
@pytest.mark.parametrize("P,ctx,window,dt", [(16, 40000, 0, BF), (128, 60001, 0, BF), (48, 30000, 0, HF), (64, 50000, 20000, BF), (16, 33000, 0, HF)])
def test_prompt(kv, P, ctx, window, dt, name):
    n = 70
    c = prompt.case(101, [n], [ctx], 4, 2, P, dt, window=window, spread=0.1)
    name_values(c["vc"], c["table"][0], n + ctx, P, CLASSES[name])
    out, lse = prompt.call(kv, c)
    j, pos = torch.arange(n + ctx, device="cuda"), ctx + torch.arange(n, device="cuda")[:, None]
    seen = (j <= pos) & ((j > pos - window) if window else True)
    kc = torch.nan_to_num(c["kc"])  # (what no row sees)
    table = torch.where(c["table"] < kc.shape[0], c["table"], 0)[0]
    want, want_lse, reach, shares, pages = oracle(c["q"], kc, [(table, n + ctx)], P, CLASSES[name], SCALE, seen)
    shown = pages < ctx // P  # pages that every row sees whole
    check(out, lse, want, want_lse, reach, n + ctx, dt, *((shares[:, :, shown], pages[shown]) if name == "page" and not window else ()))


@pytest.mark.parametrize("name", list(CLASSES))
@pytest.mark.parametrize("P,n,dt", [(16, 40000, BF), (128, 50001, BF), (48, 24000, HF)])
def test_prefix(kv, P, n, dt, name):
    tail = 5 * P
    c = prefix.case(102, [n], [3], [tail] * 3, 4, 2, P, dt, spread=0.1)
    name_values(c["vc"], c["prefix_table"][0], n, P, CLASSES[name])
    for b in range(3):
        name_values(c["vc"], c["table"][b], tail, P, CLASSES[name])
    out, lse = prefix.call(kv, c)
    for b in range(3):
        seen = torch.ones(1, n + tail, dtype=torch.bool, device="cuda")
        want, want_lse, reach, shares, pages = oracle(c["q"][b:b + 1], c["kc"], [(c["prefix_table"][0], n), (c["table"][b], tail)], P,
                                                      CLASSES[name], SCALE, seen)
        check(out[b:b + 1], lse[b:b + 1], want, want_lse, reach, n + tail, dt, *((shares, pages) if name == "page" else ()))
