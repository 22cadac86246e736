"""Order of the paged-cache kernels on a stream. Their grids may start while the grid in
front of them still runs, so what others wrote may be read behind a wait only."""
import os
import re

import pytest
import torch

bd = pytest.importorskip("block_causal_varlen_gb300")
pu = pytest.importorskip("paged_util")

CSRC = os.path.join(os.path.dirname(bd.__file__), "csrc")
WAIT = r"grid_wait\(\)|take_go\("
READ = r"\bplan\[|\brec\[|\bpieces\[|->|__ldc[gs]\(|\btma_load|\bcp\.async|\ba\.\w+\["


def kernels():
    for f in sorted(os.listdir(CSRC)):
        if not re.fullmatch(r"paged_\w+\.cu", f):
            continue
        s = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, f)).read())
        for m in re.finditer(r"__global__ void.*?(\w+_kernel)\(", s, re.S):
            at = s.index("{", s.index(") {", m.end()))
            depth, end = 0, at
            while True:
                depth += {"{": 1, "}": -1}.get(s[end], 0)
                end += 1
                if depth == 0:
                    break
            yield f, m.group(1), s[at:end]


def test_every_kernel_waits_before_its_first_read():
    names = []
    for f, name, body in kernels():
        names.append(name)
        wait = re.search(WAIT, body)
        assert wait, (f, name)
        early = re.search(READ, body[:wait.start()])
        assert early is None, (f, name, early and early.group(0))
        # what is not this wait takes a word instead, orders the copies behind it as well, and ends
        # no sooner than the grid in front of it
        if "take_go" in body:
            m = re.search(r"if constexpr \(BEHIND\) \{\s*if \(threadIdx\.x == 0\) abort_flag\[1\] = take_go\([^;]*;\s*__syncthreads\(\);\s*"
                          r"if \(!abort_flag\[1\]\) grid_wait\(\);\s*else fence_proxy_async_all\(\);\s*\} else \{\s*grid_wait\(\);\s*\}", body)
            assert m and re.search(READ, body[:m.end()]) is None, name
            assert re.search(r"if \(p0 == p1\) \{\s*if constexpr \(BEHIND\) grid_wait\(\);\s*return;", body), name
            assert body.rindex("if constexpr (BEHIND) grid_wait()") > body.rindex("for (int p = p0; p < p1; ++p)"), name
        else:
            line = body[body.rfind("\n", 0, wait.start()):wait.start()]
            assert line.strip() == "", (name, line)
    assert {"bd_cache_write_kernel", "bd_cache_read_kernel", "bd_paged_dec_kernel", "bd_paged_tile_kernel", "bd_paged_merge_kernel",
            "bd_paged_wide_merge_kernel", "bd_paged_tile_merge_kernel"} == set(names)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_few_rows_beside_tiles_whatever_the_workspace_holds(fmt):
    """A step of both kernels: the same bits over any workspace contents, and again and again
    over one workspace; the words that order the kernels are left cleared."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = pu.Case([60, 1, 200, 3], [5000, 700, 260, 90], 8, 2, 128, page=32, fmt=fmt)
    n = bd.bd_paged_attn_workspace(c.plan)
    g = torch.Generator(device="cuda").manual_seed(0)
    spaces = [torch.zeros(n, dtype=torch.uint8, device="cuda"), torch.full((n,), 255, dtype=torch.uint8, device="cuda"),
              torch.randint(0, 256, (n,), generator=g, dtype=torch.uint8, device="cuda")]
    want = None
    for ws in spaces:
        for _ in range(20):
            got = pu.run_attention(c, workspace=ws)
            if want is None:
                want = got
                pu.check_attention(c, *got)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (ws[-304 * 8:] == 0).all()
