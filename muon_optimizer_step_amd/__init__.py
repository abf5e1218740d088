"""MI355X (gfx950) Muon optimizer step, weight EMA and AdamW for the other parameters,
with the loss of the language-model head (its gradients included), AdamW on 8-bit states, and linear layers in 8 bits.

Thin Python binding over the C ABI of libmuonstep.so (include/muonstep.h, muonstep_train.h, muonstep_linear8.h):
it only turns torch tensors into device pointers plus the current HIP stream.
Every step of the computation runs in the library's HIP kernels.
"""

from ._lib import (  # noqa: F401
    MUON_NS_BF16, MUON_NS_FP32, MUON_NS_BF16X3, MUON_NS_SCHEDULE_PHASES, MUON_NS_SCHEDULE_CHAIN, MuonError, LIB_PATH,
    load, set_ns_schedule, plan_cache_stats,
)
from .api import (  # noqa: F401
    muon_step, muon_step_static, ema_update, ema_swap, adamw_step, workspace_size, profile_enable, profile_read, version,
    PreparedMuonStep, PreparedEma, PreparedAdamW,
)
from .train import (  # noqa: F401
    AdamW8State, adamw8_step, PreparedAdamW8, LinearCrossEntropy, PreparedLinearCrossEntropy, linear_cross_entropy,
    linear_cross_entropy_grad,
)
from .linear8 import (  # noqa: F401
    Activation8, Weight8, Encoded8, ActGrad8, act8_encode, act8_backward, act8_grad_weight, weight8_encode, matmul8,
    PreparedAct8Encode, PreparedAct8Backward, PreparedAct8GradWeight, PreparedWeight8Encode, PreparedMatmul8,
)
