"""MI355X (gfx950) embedding weight-gradient accumulation.

    main_grad += embedding_dense_backward(grad, ids), touching only the rows of ids

with the arithmetic of PyTorch's sort-based embedding backward followed by
main_grad.add_ (Megatron-Core API docs, "core.fusions.fused_embedding_wgrad").
Beside it, the operators of a training step that meet the same vocabulary and
the same main_grad: token_logprobs and token_logprobs_backward (the loss over
the vocabulary and the gradient the backward pass starts from),
orthogonalize_update and muon_step (an update made from main_grad,
orthogonalised and applied to the weight).
The work runs in hand-written HIP kernels behind the C ABI of
include/embedding_wgrad.h, token_logprobs.h and muon.h; this package is a thin
binding to it.
"""
from ._binding import (  # noqa: F401
    MANY_MAX_EMBEDDINGS,
    MANY_MAX_TOKENS,
    MAX_TOKENS,
    MIN_TOKENS,
    NO_ALLOC_SCRATCH_BYTES,
    NROWS,
    EmbeddingWgradError,
    WaitGaveUpError,
    accumulate_embedding_wgrad,
    accumulate_embedding_wgrad_many_tokens,
    accumulate_embedding_wgrad_no_alloc,
    accumulate_embedding_wgrad_vocab_shard,
    can_accumulate_embedding_wgrad,
    can_accumulate_embedding_wgrad_many_tokens,
    can_accumulate_embedding_wgrad_vocab_shard,
    invalid_id_count,
    many_tokens_workspace_bytes,
    new_many_tokens_workspace,
    new_workspace,
    position_bits,
    raise_if_waits_gave_up,
    sort_tokens,
    wait_timeouts,
    workspace_bytes,
)
from ._binding import LIBRARY as library_path  # noqa: F401
from ._logprobs import (  # noqa: F401
    MAX_TOP_LOGPROBS,
    TokenLogprobs,
    token_logprobs,
    token_logprobs_backward,
    token_logprobs_workspace_bytes,
)
from ._muon import (  # noqa: F401
    NEWTON_SCHULZ_COEFFICIENTS,
    muon_step,
    orthogonalize_update,
    orthogonalize_update_workspace_bytes,
)
