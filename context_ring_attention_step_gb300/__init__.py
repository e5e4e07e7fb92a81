"""GB300 (sm_103a) ring attention for context parallelism.

The compute path lives in ``libring_attn.so`` (hand-written tcgen05/TMA CUDA
kernels behind the C ABI in ``include/ring_attn.h``); this package is its
thin Python binding.
"""

from .ring_attn import (  # noqa: F401
    LAYOUTS,
    Plan,
    RingAttention,
    RingAttnError,
    dynamic_cp,
    load_library,
    ring_attn_bwd,
    ring_attn_fwd,
    ring_attention,
    workspace_status,
)
from .kv_cache import (  # noqa: F401
    Kv4Cache,
    Kv4Eviction,
    Kv4Tables,
    kv4_attention,
    kv4_attention_workspace,
    kv4_evict,
    kv4_evict_out,
    kv4_evict_workspace,
    kv4_load,
    kv4_move,
    kv4_status,
    kv4_store,
    kv4_tables,
    kv4_tables_out,
    kv4_weights,
)
from .rope import (  # noqa: F401
    QkNormRope,
    Rotary,
    qk_norm_rope,
    qk_norm_rope_bwd,
    qk_norm_rope_fwd,
    qk_norm_rope_workspace,
    rope_positions,
)
