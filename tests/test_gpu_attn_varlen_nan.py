"""NaN and infinities inside a sequence of the packed attention: they reach the rows that see them, in O, in the
log-sum-exp and in the gradients, whichever form of the kernels computes a row (a CTA alone, or a cluster that shares its
keys). Everything else is compared bit for bit with the same call on clean inputs."""
import pytest
import torch

from test_gpu_attn_varlen import _cu, _inputs, _run

pytestmark = pytest.mark.gpu
NAN = float("nan")
FORMS = [([300], [300]),      # fewer than four key tiles: a CTA alone
         ([40], [4500]),      # clusters share the keys
         ([1100], [1100])]    # clusters, several query tiles


def _isnan(x):
    return torch.isnan(x.float())


def _runs(q_lens, k_lens, causal, dirty, d=64, grad=True, heads=2, kv=1):
    """Outputs on clean inputs and on the ones that `dirty` changes."""
    cu_q, cu_k = _cu(q_lens), _cu(k_lens)
    clean = _inputs(sum(q_lens), sum(k_lens), heads, kv, d, seed=24000 + sum(k_lens))
    other = {k: v.clone() for k, v in clean.items()}
    dirty(other)
    return _run(clean, cu_q, cu_k, causal, grad=grad), _run(other, cu_q, cu_k, causal, grad=grad)


@pytest.mark.parametrize("q_lens,k_lens", FORMS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_nan_in_a_query(q_lens, k_lens, causal, d):
    # one row of one head: its O, log-sum-exp and dQ are NaN, and all other rows' as without it
    row = 5

    def dirty(x):
        x["Q"][row, 0] = NAN

    a, b = _runs(q_lens, k_lens, causal, dirty, d)
    assert torch.isnan(b["LSE"][0, row]) and _isnan(b["O"][row, 0]).all() and _isnan(b["dQ"][row, 0]).all()
    for k in ("O", "dQ", "LSE"):
        at = (0, row) if k == "LSE" else (row, 0)
        b[k][at] = a[k][at]
        assert torch.equal(a[k], b[k]), k


@pytest.mark.parametrize("q_lens,k_lens", FORMS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("value", [NAN, float("inf")])
def test_nan_in_a_key(q_lens, k_lens, causal, value):
    # rows that see the key carry the NaN; rows from which it is hidden are as without it. (Infinite in every element:
    # scores of both signs of infinity summed, so NaN too.)
    nq, nk = q_lens[0], k_lens[0]
    key = nk - nq // 2

    def dirty(x):
        x["K"][key] = value

    a, b = _runs(q_lens, k_lens, causal, dirty, grad=False)
    first = key - (nk - nq) if causal else 0
    assert torch.isnan(b["LSE"][:, first:]).all() and _isnan(b["O"][first:]).any(-1).all()
    assert torch.equal(b["LSE"][:, :first], a["LSE"][:, :first]) and torch.equal(b["O"][:first], a["O"][:first])


@pytest.mark.parametrize("q_lens,k_lens", FORMS)
def test_scores_of_minus_infinity(q_lens, k_lens):
    # a key at minus infinity has no weight; a row that sees only such keys has none to give: O = 0, LSE = -inf
    nq, nk = q_lens[0], k_lens[0]

    def dirty(x):
        x["Q"][:, :, 0] = 1.0
        x["Q"][3, :, 0] = 2.0
        x["K"][0, :, 0] = -float("inf")

    a, b = _runs(q_lens, k_lens, False, dirty, grad=False)
    assert torch.isfinite(b["O"].float()).all() and torch.isfinite(b["LSE"]).all()

    def all_keys(x):
        x["Q"][:, :, 0] = 1.0
        x["K"][:, :, 0] = -float("inf")

    _, b = _runs(q_lens, k_lens, False, all_keys, grad=False)
    assert torch.isneginf(b["LSE"]).all() and not b["O"].any()


@pytest.mark.parametrize("q_lens,k_lens", [
    ([200], [70]),           # 130 rows without keys: a whole tile, and two of the next
    ([2300], [2200]),        # 100, where clusters share keys and queries
    ([90, 300, 5], [40, 171, 0]),
])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_rows_without_keys_give_nothing(q_lens, k_lens, d):
    # causal rows before the first key: whatever their Q and dO hold, no gradient comes from them
    cu, at = _cu(q_lens), []
    for i, (nq, nk) in enumerate(zip(q_lens, k_lens)):
        at += range(int(cu[i]), int(cu[i]) + (nq if nk == 0 else max(0, nq - nk)))

    def dirty(x):
        x["Q"][at[0::2]] = NAN
        x["Q"][at[1::2]] = float("inf")
        x["dO"][at[0::3]] = float("inf")
        x["dO"][at[1::3]] = NAN

    a, b = _runs(q_lens, k_lens, True, dirty, d)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    assert not b["O"][at].any() and not b["dQ"][at].any() and torch.isneginf(b["LSE"][:, at]).all()


@pytest.mark.parametrize("q_lens,k_lens", [([200], [70]), ([2300], [2200])])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_rows_without_keys_stay_zero_beside_a_nan_key(q_lens, k_lens, d):
    # K and V of a key in the tile that such rows' products run over
    nq, nk = q_lens[0], k_lens[0]

    def dirty(x):
        x["K"][2] = NAN
        x["V"][2] = float("inf")

    _, b = _runs(q_lens, k_lens, True, dirty, d)
    dead = nq - nk
    assert not b["O"][:dead].any() and not b["dQ"][:dead].any() and torch.isneginf(b["LSE"][:, :dead]).all()


@pytest.mark.parametrize("q_lens,k_lens,heads,kv", [
    ([40, 30, 5], [4500, 4333, 3000], 2, 1),     # clusters share the keys (forward, dQ)
    ([900, 130, 77], [900, 130, 77], 8, 1),      # clusters share the queries (dK, dV)
])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_other_sequences_do_not_leak_through_clusters(q_lens, k_lens, heads, kv, causal, d):
    # the second sequence is all NaN, the third infinite: the first is as without them
    nq, nk = q_lens[0], k_lens[0]

    def dirty(x):
        for k, v in x.items():
            lens = k_lens if k in ("K", "V") else q_lens
            v[lens[0]:lens[0] + lens[1]] = NAN
            v[lens[0] + lens[1]:] = float("inf")

    a, b = _runs(q_lens, k_lens, causal, dirty, d, heads=heads, kv=kv)
    for k in a:
        sl = (slice(None), slice(0, nq)) if k == "LSE" else slice(0, nk if k in ("dK", "dV") else nq)
        assert torch.equal(a[k][sl], b[k][sl]), k
