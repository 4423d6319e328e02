"""Which calls of attention over 4 bits cut their requests into runs: those that join them launch twice (CPU only)."""
import pytest

from tests.test_cache4_host import walk4
from tests.test_verify_host import runtime  # noqa: F401

# heads, dim, requests, tokens, bound on the keys, cut: both sides of the rule as they were timed
CALLS = [
    ((32, 8), 128, 1, 1, 1024, False), ((32, 8), 128, 1, 1, 2048, True), ((32, 8), 128, 12, 1, 2048, False),
    ((32, 8), 128, 12, 1, 4096, True), ((32, 8), 128, 20, 8, 1536, False), ((32, 8), 128, 20, 8, 2048, True),
    ((32, 8), 128, 32, 8, 2048, False), ((32, 8), 128, 32, 8, 4096, True), ((32, 8), 128, 64, 8, 16384, False),
    ((32, 8), 64, 1, 1, 1536, False), ((32, 8), 64, 4, 1, 4096, True), ((32, 8), 64, 16, 1, 2560, False),
    ((32, 8), 64, 16, 1, 6144, True), ((16, 8), 256, 4, 1, 512, False), ((16, 8), 256, 4, 1, 1024, True),
    ((16, 8), 256, 16, 8, 1024, False), ((16, 8), 256, 16, 8, 1536, True),
]


@pytest.mark.parametrize("heads,dim,requests,new,keys,cut", CALLS)
def test_requests_are_cut_where_it_pays(runtime, heads, dim, requests, new, keys, cut):  # noqa: F811
    walk4(runtime, f"""
        st, h = attention4(*{heads}, dim={dim}, requests={requests})
        assert st == 0
        c = cache4(dim={dim}, hk={heads[1]}, requests={requests}, tokens={requests * new}, max_new={new}, kv={keys}, table_width=4096,
                   table_stride=4096)
        args = (P, {heads[0] * dim}, {dim}, 0, 0, 0.1, P, {heads[0] * dim}, {dim}, None, None)
        assert lib.domino_attention_run(h, c, *args) == 0
        assert rt.host_launches() == {2 if cut else 1}
        """)
