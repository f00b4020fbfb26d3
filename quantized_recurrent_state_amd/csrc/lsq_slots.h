// Interface between the host API (lsq_api.cpp) and the slot kernels
// (lsq_slots.hip, lsq_attend.hip).  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lsq {

enum { IO_F32 = 0, IO_F16 = 1, IO_BF16 = 2 };

// Whether a launch of so many workgroups is within a launch's 2^32 - 1 threads.
inline bool fits_launch(int64_t blocks, int threads) { return blocks <= (int64_t)UINT32_MAX / threads; }

// A packed token batch over the slots of one fp32 handle (include/lsq.h,
// lsq_token_batch).
struct SlotArgs {
  float* S;                // [nslots][heads][dv][dk]
  const void* q;           // [tokens][qk_heads][dk], rows q_stride elements apart
  const void* k;
  const void* v;           // [tokens][heads][dv]
  const float* alpha;      // [tokens][heads] or [tokens][heads][dk]
  const float* beta;       // [tokens][heads]
  void* o;                 // [tokens][heads][dv]
  const int32_t* cu;       // [seqs + 1]; null: entry i is token i
  const int32_t* slots;    // [seqs]; null: entry i is slot i
  const uint8_t* fresh;    // [seqs]; null: none
  int64_t q_stride, k_stride, v_stride, o_stride;
  int64_t tokens;
  int32_t seqs, nslots, heads, share, dv;   // share: value heads per q/k head
};

// Chunked attention: the batch, its cut into segments and the workspace.
struct AttendArgs {
  SlotArgs s;
  int64_t seg_len;         // tokens per segment, a multiple of 64; 0: whole sequences
  int64_t segments, cut;   // upper bounds of their number, and of those of cut sequences
  float* ws;               // [cut][heads][dv][dk], then ws_decay (null without segments)
  float* ws_decay;         // [cut][heads]
  int32_t slices;          // workgroups over a head's value columns
  int32_t wide;            // rows of v and o begin at dwords
};

struct AttendPlan {
  int64_t seg_len, segments, cut, state_bytes;
  size_t workspace;        // bytes
  int32_t slices;
};

AttendPlan attend_plan(int64_t tokens, int32_t seqs, int32_t heads, int32_t dk, int32_t dv, int io);

// Slots copied between an fp32 handle and a quantised one (same heads, dv, dk).
struct CopyArgs {
  float* S;                // [S slots][heads][dv][dk]
  uint8_t* codes;          // [slots][heads][dv][dk*bits/8]
  void* scales;            // [slots][heads][dv][dk/group] in the stored format, or [slots][heads]
  float* ref;              // the yoked reference, or null
  const int32_t* dst_slots;
  const int32_t* src_slots;
  int32_t count, dst_n, src_n;   // entries; slots of each handle
  int32_t heads, dv, group, sfmt;
  int32_t nt;              // the read-back states take the non-temporal hint
};

hipError_t launch_walk(const SlotArgs& a, int io, int dk, int delta, int diag, int nt, hipStream_t s);
hipError_t launch_attend(const AttendArgs& a, int io, int dk, hipStream_t s);
hipError_t launch_store_slots(const CopyArgs& a, int bits, int dk, hipStream_t s);
hipError_t launch_load_slots(const CopyArgs& a, int bits, int dk, hipStream_t s);

}  // namespace lsq
