"""Batched draft verification for speculative decoding on GB300 (sm_103a).

The compute runs in the CUDA library libspecverify.so (C ABI in
include/spec_verify.h and spec_logits.h); this package only builds it and marshals arguments.
"""

from .api import (  # noqa: F401
    CascadePlan, ChainPlan, ChainPlanNoAlloc, ClaspPlan, LmHeadChainPlan, PipelineAsyncPlan, PipelinePlan,
    TreePlan,
    clasp_layer_select, compact_tree_path, verify_cascade, verify_chain, verify_pipeline, verify_pipeline_async,
    verify_tree, workspace_bytes,
)
from .logits import (  # noqa: F401
    Int4ProductPlan, ProcessLogitsPlan, QuantizeInt4Plan, int4_product, process_logits, quantize_int4,
)
from ._lib import (  # noqa: F401
    ERR_INTERNAL, ERR_MASK, ERR_NONFINITE, ERR_PARENT, ERR_TOKEN, ERR_WINDOW, ERR_ZERO_MASS,
)
from .build import build as build_library, lib_path  # noqa: F401
