"""LLM.int8() mixed-precision decomposed matmul for AMD Instinct MI355X (gfx950).

    Y = X_O . W_O (fp16) + dequant(int8(X_R) . int8(W_R))

The computation lives in hand-written HIP kernels behind a C ABI
(``include/int8mm.h``, built into ``libint8mm.so``); this package is the thin
Python binding over it, with torch used only for device memory and streams.

    import int8_quantized_matmul_col_amd as mm
    Wq, w_scale = mm.int8_prepare_weight(W)          # once per weight
    Y = mm.int8_matmul(X, Wq, w_scale, threshold=6.0)
    Y = mm.int8_linear(X, Wq, w_scale, bias)          # with a layer's bias

``Int8Linear`` wraps the same calls as a torch module (forward only), and
``replace_linear_with_int8`` swaps the fp16 ``nn.Linear`` layers of a model
for it.  ``outlier_stats`` summarizes the column maxima of an activation
(``int8_column_absmax``) and |O| at candidate thresholds
(``int8_outlier_counts``) to help choose the threshold.

Beside the matmul stand the other operators of a decode step (``serving``,
``include/int8mm_serving.h``): ``int4_linear`` (few rows times 4-bit weights
with group scales; ``Int4Linear`` is its module), and a paged key-value cache
(``PagedKVCache``) with ``kv_append``, ``kv_gather``, ``kv_attention``,
``kv_attention_shared`` (a batch that shares a prompt) and the upkeep of its
pages, ``kv_pages_reserve``, ``_extend`` (with the token maps of a batch),
``_copy``, ``_fork``, ``_free`` and ``_compact``; ``qk_rope`` turns queries and
keys by their positions, with their norms (``rotary`` prepares the frequencies),
and ``sample_tokens`` draws the next tokens.
"""

from .binding import (  # noqa: F401
    DEFAULT_THRESHOLD,
    INT8MM_DECODE_MAX_M,
    INT8MM_MAX_K,
    Int8mmError,
    int8_column_absmax,
    int8_linear,
    int8_matmul,
    int8_matmul_noalloc,
    int8_matmul_noalloc_max_workspace,
    int8_matmul_profiled,
    int8_matmul_stages,
    int8_matmul_workspace_size,
    int8_outlier_counts,
    int8_pack_weight,
    int8_prepare_weight,
    int8_weight_bytes,
    int8_weight_ld,
    padded_rows,
    unpack_weight,
    untile,
    load,
    workspace_for,
)
from .kv_cache import PagedKVCache  # noqa: F401
from .linear import Int8Linear, replace_linear_with_int8  # noqa: F401
from .linear4 import Int4Linear  # noqa: F401
from .rope import Rotary, qk_rope, rope_prepare, rotary, rotary_frequencies  # noqa: F401
from .sampling import sample_tokens, sample_tokens_workspace_size  # noqa: F401
from .stats import outlier_stats, suggest_threshold  # noqa: F401
from .serving import (  # noqa: F401
    INT8MM_KV_BAD_ROW,
    INT8MM_KV_DONE,
    INT8MM_KV_NO_PAGES,
    BatchPlan,
    Int4Weight,
    PagedKV,
    int4_linear,
    int4_linear_workspace_size,
    int4_pack_weight,
    int4_prepare_weight,
    int4_unpack_weight,
    kv_append,
    kv_attention,
    kv_attention_shared,
    kv_attention_shared_workspace_size,
    kv_attention_workspace_size,
    kv_gather,
    kv_pages_compact,
    kv_pages_copy,
    kv_pages_extend,
    kv_pages_fork,
    kv_pages_free,
    kv_pages_reserve,
)
