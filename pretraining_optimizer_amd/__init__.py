"""MI355X (gfx950) MuonH optimizer step: HIP kernels behind a C ABI.

The library (libmuonh.so, built from csrc/ by ``build.py``) runs momentum,
quintic Newton-Schulz on a grouped bf16/fp32 MFMA GEMM engine and the
Hyperball update of Eq. (1) of "Puro-2B: Poor Lab's Qwen2-1.5B Trained on
RTX 5090 within $5090" (arXiv HTML §3.3), plus the AdamW step of the
parameters MuonH does not wrap, and the operators whose gradients these steps
take: block-scaled FP8 products (§3.2), the norms, the residual's with FP8
output, attention over packed sequences and the embedding, each with its
gradient.  ``muonh`` and ``operators`` are its ctypes binding.
"""

from .muonh import (  # noqa: F401
    AdamW,
    MuonH,
    MuonHError,
    NOALLOC_MAX_WORKSPACE,
    adamw_default_options,
    default_options,
    load_library,
    plan_query,
    step_noalloc,
    workspace_size,
    MUONH_BF16,
    MUONH_F32,
    MUONH_MODE_HYPERBALL,
    MUONH_MODE_MUON_WD,
    MUONH_MODE_ELR_ALIGNED,
)
from .operators import (  # noqa: F401
    Fp8Matrix,
    add_norm_backward,
    add_norm_quantize,
    attention_backward,
    attention_forward,
    embedding_backward,
    embedding_forward,
    fp8_matmul,
    fp8_quantize,
    norm_backward,
    norm_forward,
)
