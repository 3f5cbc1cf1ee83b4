// Layout of the AdamW plan: a table of the tensors, then one entry per chunk of kAdamChunk
// elements of a tensor, tensors in order.  Written by the host, read by the kernel.
#pragma once

#include <stdint.h>

#include "../../include/bsfp8.h"

namespace bsfp8 {

constexpr int64_t kAdamChunk = 2048;  // elements of a workgroup's turn: whole 128-element blocks

typedef bsfp8_adamw_tensor AdamTensor;

struct AdamChunk {
  int32_t tensor, index;
};

inline int64_t adam_table_bytes(int64_t tensors) { return (tensors * (int64_t)sizeof(AdamTensor) + 15) / 16 * 16; }
inline int64_t adam_chunks_of(int64_t numel) { return (numel + kAdamChunk - 1) / kAdamChunk; }

}  // namespace bsfp8
