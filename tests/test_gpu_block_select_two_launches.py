"""The choice of blocks where a group's bounds do not fit on chip: scoring and selecting in a launch each, over a workspace."""
import pytest
import torch

import grouped_differential_attention_gb300 as gda
from tests.test_gpu_block_select import check, make, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from grouped_differential_attention_gb300 import build
    build.build()


@pytest.mark.parametrize("hs,hn,d,most,page,lens,keep,first,last", [
    (3, 1, 64, 32768, 0, [32768 * 16], 300, 1, 1),                       # four warps to a head
    (7, 1, 64, 25000, 0, [25000 * 16 - 5], 64, 0, 2),                    # two
    (127, 1, 64, 2600, 0, [2600 * 16], 9, 4, 0),                         # the most heads, several rounds of warps
    (6, 2, 128, 32768, 64, [32768 * 16, 201 * 16 + 3], 1000, 1, 1),      # groups, pages, long and short sequences
    (14, 2, 128, 25000, 48, [17, 0, 24999 * 16, 256 * 16, 257 * 16], 8, 0, 0),
])
def test_equals_the_reference(hs, hn, d, most, page, lens, keep, first, last):
    assert gda.gda_block_select_workspace_size(len(lens), most, hs, hn) > 0
    gda.gda_device_error(clear=True)
    check(make(len(lens), most, hs, hn, d, 16, lens, seed=hs, page=page), keep, first, last)
    assert gda.gda_device_error(clear=True) == 0


def test_equal_scores_go_to_the_lowest():
    c = make(1, 25000, 7, 1, 64, 16, [25000 * 16 - 3], seed=3, coarse=True)
    check(c, 257)


def test_replayed_over_a_workspace_of_anything_and_beside_another():
    """Outputs and workspace of the caller, whatever they held; two captured calls at once with a workspace each."""
    B, most, hs, hn, keep = 3, 2600, 127, 1, 40
    lens = [most * 16, 30 * 16, 2000 * 16 + 1]
    c = make(B, most, hs, hn, 64, 16, lens, seed=9, page=64)
    want = [t.clone() for t in run(c, keep)]
    dev = [t.cuda() for t in (*c["q"], *c["bounds"], *c["scales"], c["lens"], c["table"])]
    need = gda.gda_block_select_workspace_size(B, most, hs, hn)
    assert need > 0
    with pytest.raises(gda.GDAError):
        run(c, keep, workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    calls = []
    for _ in range(2):
        out = (torch.empty(B, hn, keep, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"))
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            gda.gda_block_select(*dev[:7], 16, keep, block_table=dev[7], out=out, workspace=ws)
        calls.append((out, ws, graph, stream))
    for fill in (0xFF, 0x7F, 0):                                         # NaN, large numbers, zeros
        for out, ws, _, _ in calls:
            ws.fill_(fill)
            for t in out:
                t.fill_(77)
        for *_, graph, stream in calls:
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                graph.replay()
        for *_, stream in calls:
            torch.cuda.current_stream().wait_stream(stream)
        for out, *_ in calls:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
