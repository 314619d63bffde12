// Layout of the 4-bit key/value cache, shared by the kernels that write, read and thin it
// (kv4.cu) and the decode kernel (decode_kv4.cu).
//
// A cache is [B][Hkv][capacity / 64] blocks of 64 consecutive slots (tokens) of one key/value
// head.  A block is one contiguous piece of 72 d bytes, so that one bulk copy brings it on chip:
//   K codes  [64][d / 2] bytes   channel 2i in bits 0-3, channel 2i + 1 in bits 4-7
//   V codes  [64][d / 2] bytes
//   K params [64][d / 64]        one 32-bit word per group of 64 channels of a row:
//   V params [64][d / 64]        fp16 step in the low half, fp16 middle in the high half
// A code c of a group stands for middle + step (c - 8).
#pragma once
#include <cuda_fp16.h>
#include <cstdint>

namespace fa {

constexpr int kKv4Block = 64;       // slots per block
constexpr int kKv4Group = 64;       // channels that share a step and a middle
constexpr float kKv4Limit = 32768.f;  // largest magnitude the format holds
constexpr uint32_t kKv4NanParam = 0x7E007E00u;  // step = middle = NaN: the group reads as NaN

__host__ __device__ constexpr int kv4_block_bytes(int d) { return 72 * d; }
__host__ __device__ constexpr int kv4_code_bytes(int d) { return d / 2; }       // of a row
__host__ __device__ constexpr int kv4_param_words(int d) { return d / 64; }     // of a row
// byte offsets inside a block; which: 0 keys, 1 values
__host__ __device__ constexpr int kv4_codes_at(int d, int which) { return which * 32 * d; }
__host__ __device__ constexpr int kv4_params_at(int d, int which) { return 64 * d + which * 4 * d; }

}  // namespace fa
