"""Host-side checks at the limits of what the operators around a prefix cache allow (no GPU: no call here reaches a kernel)."""
from test_ops_host import NULL, _call, _i, _z, gdn  # noqa: F401
from test_prefix_host import _sample, _shared


def test_a_prefix_without_cached_tokens_needs_its_pages(gdn):  # noqa: F811
    # no token is cached yet, but prefix_len may be up to max_prefix_len: its pages would be read
    for i in (1, 2, 3):
        assert _call(gdn, "gdn_shared_attn", _shared(gdn, max_kv_len=0, max_prefix_len=32, max_own_len=0), 10, {i: None}, ws_bytes=255) == NULL, i
        assert _call(gdn, "gdn_shared_attn", _shared(gdn, max_kv_len=0, max_prefix_len=1), 10, {i: None}, ws_bytes=255) == NULL, i


def test_bounds_of_a_prefix_beyond_every_kv_len(gdn):  # noqa: F811
    q, kc, table = _z(2, 8, 128), _z(10, 16, 2, 128), _i(1, 2, 3, 4, 5, 6).view(2, 3)

    def bounds(**kw):
        d = gdn.make_shared_desc(q, kc, table, 2, 1, **kw)
        return d.cache.max_kv_len, d.max_prefix_len, d.max_own_len

    assert bounds() == (48, 48, 48) and bounds(max_kv_len=35) == (35, 35, 35)
    assert bounds(max_kv_len=35, max_prefix_len=40) == (35, 40, 35)
    assert bounds(max_kv_len=35, max_prefix_len=100, max_own_len=40) == (35, 48, 35)      # as much as a table's row holds
    assert bounds(max_kv_len=0, max_prefix_len=40, max_own_len=0) == (0, 40, 0)
    assert bounds(max_kv_len=1 << 30, max_prefix_len=1 << 30, max_own_len=7) == (48, 48, 7)


def test_sample_workspace_serves_fewer_rows(gdn):  # noqa: F811
    for dtype in (0, 1):
        for vocab in (1, 100, 2049, 8192, 8193, 32000, 49999, 65536, 65537, 131072, 1 << 24):
            need = [gdn.gdn_sample_workspace_bytes(_sample(gdn, rows=r, vocab=vocab, stride=vocab, dtype=dtype)) for r in range(0, 500)]
            assert need == sorted(need), (dtype, vocab)
