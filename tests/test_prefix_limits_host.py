"""Host-side checks at the limits of what the operators around a prefix cache allow (no GPU: no call here reaches a kernel)."""
from test_ops_host import NULL, _call, gdn  # noqa: F401
from test_prefix_host import _shared


def test_a_prefix_without_cached_tokens_needs_its_pages(gdn):  # noqa: F811
    # no token is cached yet, but prefix_len may be up to max_prefix_len: its pages would be read
    for i in (1, 2, 3):
        assert _call(gdn, "gdn_shared_attn", _shared(gdn, max_kv_len=0, max_prefix_len=32, max_own_len=0), 10, {i: None}, ws_bytes=255) == NULL, i
        assert _call(gdn, "gdn_shared_attn", _shared(gdn, max_kv_len=0, max_prefix_len=1), 10, {i: None}, ws_bytes=255) == NULL, i
