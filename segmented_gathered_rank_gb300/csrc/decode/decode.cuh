// Shared by the decode-step operators: host-side checks of the paged cache and
// the device view of one request's cached tokens.
#pragma once

#include "internal.cuh"

namespace lora {
namespace decode {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxPageSize = 1024;

// Host checks shared by the calls on a paged cache.
inline int check_kv(const lora_kv_pages *kv, int n_q_heads) {
    if (!kv || !kv->k || !kv->v || (kv->dtype != LORA_F32 && kv->dtype != LORA_BF16)) return LORA_ERR_ARG;
    if (!aligned16(kv->k) || !aligned16(kv->v) || ((uintptr_t)kv->status & 3u)) return LORA_ERR_ARG;
    if (kv->n_pages < 1 || kv->n_kv_heads < 1 || n_q_heads < 0) return LORA_ERR_ARG;
    if (kv->page_size < 1 || kv->page_size > kMaxPageSize || (kv->page_size & (kv->page_size - 1))) return LORA_ERR_SHAPE;
    if (kv->head_dim < 8 || kv->head_dim > kMaxHeadDim || kv->head_dim % 8) return LORA_ERR_SHAPE;
    if (n_q_heads % kv->n_kv_heads) return LORA_ERR_SHAPE;
    if ((long long)kv->n_pages * kv->page_size > 0x7fffffffLL / kv->n_kv_heads) return LORA_ERR_SHAPE;   // rows are ints
    return LORA_OK;
}

inline int log2_of(int power_of_two) {
    int n = 0;
    while ((1 << n) < power_of_two) ++n;
    return n;
}

__device__ __forceinline__ void flag_status(int *status, int bits) {
    if (status) atomicOr(status, bits);
}

// One lane of a converged warp.  The compiler knows that a branch on it has one
// thread, so that the operands of tcgen05 instructions inside, which the hardware
// wants uniform, need no loop over lanes (32 against 57 cycles a 128 x 64 x 16
// product measured, for `lane == 0`).
__device__ __forceinline__ bool elect_lane() {
    uint32_t mine = 0;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\n@p mov.s32 %0, 1;\n}\n" : "+r"(mine));
    return mine != 0;
}

}  // namespace decode
}  // namespace lora
