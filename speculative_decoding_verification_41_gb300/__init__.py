"""libdspark: GB300-native batched speculative verification and the
hardware-aware prefix scheduler of DSpark, and its drafter's sequential stage
with the Markov head, behind a C-ABI (include/dspark.h), and the paged
key-value cache around a step: pages, append and attention
(include/dspark_paged.h). Python calls go through `binding` (ctypes) and
`paged` (a small C++ module, csrc/paged_binding.cpp, and ctypes), which check and
marshal arguments only; `paged_q8` the same cache in 8
bits and rotary positions (include/dspark_q8.h); `paged_step` runs a whole step on the paged cache;
`workloads` generates seeded synthetic inputs."""
from .binding import (DsparkError, ScheduleBuffers, VerifyBuffers, dspark_draft_markov,  # noqa: F401
                      dspark_schedule, dspark_verify, draft_workspace_bytes,
                      schedule_workspace_bytes, verify_workspace_bytes)
from .paged import (AttentionBuffers, ReleaseBuffers, ReserveBuffers,  # noqa: F401
                    dspark_kv_append, dspark_paged_attention, dspark_pages_release,
                    dspark_pages_reserve)
from .paged_q8 import (RotaryTable, dspark_kv_append_q8, dspark_kv_gather_q8,  # noqa: F401
                       dspark_paged_attention_q8, dspark_rotary)
