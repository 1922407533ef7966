"""Calls of masked attention whose CTAs take two query tiles each (more pairs of a head and a query tile than SMs),
and calls whose grid is walked head by head although they are causal.  Shared by the host test that asserts
this from the plan and the GPU tests that run them."""

# name: (batch, n_q, n_k, heads_q, heads_kv, head_dim, rule); rule: letters of `rule_of`
TWO_TILES = {
    "plain": (2, 700, 700, 20, 20, 64, ""),
    "plain_128_odd_tiles": (1, 300, 520, 52, 52, 128, ""),
    "causal": (2, 700, 700, 20, 20, 64, "c"),
    "causal_128_odd_tiles": (1, 300, 520, 52, 52, 128, "c"),
    "causal_more_queries_than_keys": (1, 700, 300, 40, 20, 64, "c"),
    "prefix": (2, 390, 400, 24, 12, 72, "cp"),
    "documents": (2, 700, 700, 20, 20, 64, "d"),
    "documents_128": (1, 520, 520, 40, 10, 128, "d"),
    "documents_causal_odd_tiles": (2, 333, 600, 28, 14, 72, "cd"),
    "cap": (2, 700, 700, 20, 20, 64, "k"),
    "bias": (2, 390, 500, 20, 20, 72, "b"),
    "cap_bias_prefix_documents": (2, 700, 700, 20, 20, 64, "kbcpd"),
    "cap_bias_causal_128": (1, 300, 300, 52, 52, 128, "kbc"),
    "packed_4": (40, 40, 150, 8, 2, 64, "c"),
    "packed_3_last_rows_unwritten": (40, 50, 290, 6, 2, 64, "kb"),
    "packed_3_odd_tiles": (16, 200, 300, 6, 2, 128, "cd"),
    "packed_5_documents": (40, 30, 200, 10, 2, 72, "d"),
}
# name: (query heads per tile, query tiles of a head or of the heads that share a key head)
LAYOUT = {
    "plain": (1, 6), "plain_128_odd_tiles": (1, 3), "causal": (1, 6), "causal_128_odd_tiles": (1, 3),
    "causal_more_queries_than_keys": (2, 11), "prefix": (2, 7), "documents": (1, 6), "documents_128": (4, 17),
    "documents_causal_odd_tiles": (1, 3), "cap": (1, 6), "bias": (1, 4), "cap_bias_prefix_documents": (1, 6),
    "cap_bias_causal_128": (1, 3), "packed_4": (4, 2), "packed_3_last_rows_unwritten": (3, 2),
    "packed_3_odd_tiles": (3, 5), "packed_5_documents": (5, 2),
}
# many heads over long keys: K and V of all heads together are larger than L2
HEAD_BY_HEAD = {
    "causal_64": (1, 200, 6000, 80, 80, 64, "c"),
    "causal_128_prefix": (1, 150, 6000, 120, 60, 128, "cp"),
}
# few pairs: the keys are split over a cluster
SPLIT = {
    "one_query_one_head": (1, 1, 1100, 1, 1, 64, ""),
    "one_query_72": (1, 1, 1100, 2, 2, 72, ""),
    "one_query_shared_heads": (1, 1, 1100, 6, 2, 128, ""),
}
