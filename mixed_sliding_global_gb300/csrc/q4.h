// q4.h -- launch interfaces of the 4-bit KV cache kernels.
//
// Format of a cache row (one position of one KV head, head_dim elements): groups of 64 elements
// share a scale s, the smallest number of at most five significant bits (at least 2^-126) with
// 7 s >= max |x| (at most 1.125 * 2^125, so that 7 s is finite in bf16; 0 for a group of zeros,
// NaN for a group holding a NaN or an infinity); each
// element is a code rint(x / s) in [-7, 7]. Three plus five significant bits: code * s is exact
// in bf16. Codes are sign-magnitude, eight to a 32-bit word: element 2j has its magnitude in bits
// 4j..4j+2 and its sign in bit (15 + 4j) % 32, element 2j + 1 in bits 16+4j..16+4j+2 and bit
// (31 + 4j) % 32. So rotr(word, 4j) & 0x80078007 is the pair of elements 2j, 2j + 1 as two fp16
// numbers code * 2^-24 (subnormals, which the tensor cores multiply exactly): two instructions
// per pair and no conversion.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "attn_internal.h"

namespace gemma {

constexpr int kQ4Group = 64;  // elements per scale

// Where the rows of an owner layer's 4-bit cache live (block_table == nullptr: a plain cache, or
// a ring of `ring` slots).
struct Q4Cache {
    uint8_t* k_codes;        // [rows][slots][head_dim / 2]
    __nv_bfloat16* k_scales; // [rows][slots][head_dim / 64]
    uint8_t* v_codes;        // nullptr when K serves as V
    __nv_bfloat16* v_scales;
    int n_kv, cap, ring;
    PagedLayout pg;
};

// Attention of a few query rows straight over the cache (q4_attn.cu) by C CTAs: with `balanced`
// each takes an equal share of the launch's key tiles (parts of units meet in p.o_part
// [C][2][row tile][head_dim] and p.ml_part [C][2][row tile][2], with two ints per unit in info, and
// are merged by a second launch), else `cluster` CTAs (a cluster, which merges its parts through
// distributed shared memory) take a unit (sequence, KV head, row tile) and C counts all of them.
constexpr int kQ4KeyTile = 128;
constexpr int kQ4CtasPerSm = 2;
constexpr int kQ4MaxShares = 512;  // C of a balanced launch
constexpr int kQ4MaxCluster = 8;
// rows (token, query head) per CTA
inline int q4_row_tile(int rows) { return rows > 8 ? 16 : 8; }
cudaError_t launch_q4_attn(const RowsParams& p, const Q4Cache& c, int head_dim, int batch, int C,
                           int balanced, int cluster, void* info, cudaStream_t st);

cudaError_t launch_q4_append(const Q4Cache& c, const void* k_new, const void* v_new,
                             const int32_t* write_pos, int batch, int n_new, int head_dim,
                             int fp32, uint32_t* err, int n_sm, cudaStream_t st);

// Dequantised rows read_pos[b] + t, t < n_rows, as [batch][n_rows][n_kv][head_dim].
cudaError_t launch_q4_read(const Q4Cache& c, void* k_out, void* v_out, const int32_t* read_pos,
                           int batch, int n_rows, int head_dim, int fp32, uint32_t* err, int n_sm,
                           cudaStream_t st);

// Dequantise the positions a step of n_tok queries may read (from the first query's window start
// to the last position) into a bf16 cache [batch][n_kv][slots][head_dim] whose slot 0 is that
// first position, and write the sequences' lengths in that numbering (0 for an invalid one).
cudaError_t launch_q4_expand(const Q4Cache& c, void* k_out, void* v_out, int32_t* lens_out,
                             const int32_t* seq_lens, int batch, int n_tok, int max_seq_len,
                             int window, int slots, int head_dim, uint32_t* err, int n_sm,
                             cudaStream_t st);

}  // namespace gemma
