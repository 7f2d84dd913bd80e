"""GB300-native (sm_103a) per-layer MoE expert path of Specter's Streamlined
Execution Engine: routing, expert-activation counters, gather by expert, the
fused INT4 draft MLP, the expert-reordered FP16 verify MLP, the shared expert
and the weighted combine, with latent attention over a paged cache, its append
and the verify logits' log probabilities around it, and, for models with ordinary keys
and values, trees of drafted tokens, their append, attention and acceptance over a paged
cache, as hand-written CUDA behind the C ABI in include/spx.h (libspx.so).  ``spx`` is the thin Python binding."""
from . import build  # noqa: F401
