"""awq_kv4_attention_workspace_bytes with max_kv = 0, without a GPU: the call with max_kv = 0 splits its work by what the table can hold,
which the query does not know, so the query's answer has to be enough for every table. No call here reaches the device: each one is
given a workspace that is not aligned, which is looked at after its size."""
import pytest

from test_attn_abi_cpu import FAKE, UNSUPPORTED, WORKSPACE, _attend, _err, lib  # noqa: F401


@pytest.mark.parametrize("n,seqs,heads,kv,d,causal,window,ragged", [
    (1, 1, 64, 8, 128, 1, 0, False), (8, 4, 4, 2, 64, 1, 0, False), (24, 4, 16, 8, 256, 1, 2048, True), (4, 4, 32, 32, 128, 0, 100, False),
    (300, 1, 8, 2, 128, 1, 0, False), (200, 2, 2, 1, 224, 0, 0, True)])
def test_a_query_without_max_kv_is_enough_for_every_table(lib, n, seqs, heads, kv, d, causal, window, ragged):  # noqa: F811
    query = lib.awq_kv4_attention_workspace_bytes
    nb = query(n, seqs, int(ragged), heads, kv, d, causal, window, 0)
    assert nb == max(query(n, seqs, int(ragged), heads, kv, d, causal, window, 1 << e) for e in range(31)) > 0
    groups, page = (d + 127) // 128, 64
    rows = 2 * kv * page
    needed = 0
    for width in (1, 5, 50, 1000, 30000, 1 << 24):
        kw = dict(n=n, seqs=seqs, heads=heads, kv=kv, d=d, ld_q=heads * d, ld_q_head=d, ld_out=heads * d, ld_out_head=d, causal=causal, window=window,
                  q_offsets=FAKE if ragged else None, page=page, page_codes=rows * d // 2, page_params=rows * groups, width=width,
                  ld_table=width, max_kv=0, out=FAKE + 0x1000000)
        need = query(n, seqs, int(ragged), heads, kv, d, causal, window, width * page)
        assert need <= nb
        # (what the table holds is past 32 bits of the split's units: no workspace is needed then)
        tiles = n * heads // kv // 16 + seqs
        if need == 0 or tiles * kv * (width * page // 128 + 1) > 0x7FFFFFFF:
            continue
        needed += 1
        assert _attend(lib, ws=FAKE + 64, nb=nb, **kw) == UNSUPPORTED, _err(lib)
        assert _attend(lib, ws=FAKE, nb=need - 1, **kw) == WORKSPACE, _err(lib)
    assert needed
