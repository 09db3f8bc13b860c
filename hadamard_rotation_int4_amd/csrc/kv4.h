// What the host side hands to the kernels of the 4-bit key/value cache.
#pragma once

#include "hr_internal.h"

namespace hr {

// Element types of the key/value cache calls (the values of hr_dtype).
constexpr int kDtF32 = 0, kDtBf16 = 1, kDtF16 = 2;

// Largest cached length: token indices of a sequence stay in 32 bits.
constexpr int kKv4MaxLen = 1 << 30;

// A 4-bit key/value cache after host validation (layout: kv4_device.h).
struct Kv4Cache {
  uint8_t* codes[2];     // keys, values
  _Float16* scales[2];
  const int8_t* signs;   // [dim] or null (all +1; only read with rotate)
  int64_t pages;
  int heads, dim, group;
  int page_log2;
  int rotate;
};

struct Kv4AppendArgs {
  Kv4Cache c;
  const void* x[2];      // keys, values: [tokens] rows of [heads][dim], rows `stride` elements apart
  int64_t stride[2];
  int dtype;
  const int64_t* slots;
  int64_t tokens;
};

struct Kv4ReadArgs {
  Kv4Cache c;
  void* y[2];            // keys, values: [tokens][heads][dim]
  int dtype;
  const int64_t* slots;
  int64_t tokens;
};

struct Kv4AttnArgs {
  Kv4Cache c;
  const void* q;         // [total] rows of [q_heads][dim], rows q_stride elements apart
  int64_t q_stride;
  int dtype;             // of q and out
  int64_t total;
  const int32_t* starts; // [batch + 1] first row of each sequence, or null (max_new rows each)
  const int32_t* table;  // [batch][width] page ids
  int64_t width;
  const int32_t* lens;   // [batch]
  int batch, q_heads, rep;
  int max_new;
  int64_t max_len;
  float scale;
  int causal, window;
  void* out;             // [total][q_heads][dim]
  float* part_o;         // [total * q_heads][nsplit][dim] sums, not yet divided; null when nsplit == 1
  float2* part_ml;       // [total * q_heads][nsplit] (running max in log2 units, sum)
  // by kv4_attention_plan:
  int rows;              // of a row tile: 16, 32, or 128 or 256 (kv4_prompt.hip)
  int waves;             // of a workgroup with 16 rows: 4 or 8
  int tiles;             // row tiles of a (sequence, key/value head)
  int nsplit, chunk;     // most parts of the token axis, tokens of a part
  int64_t groups;        // workgroups
};

hipError_t launch_kv4_append(const Kv4AppendArgs& a, hipStream_t s);
hipError_t launch_kv4_read(const Kv4ReadArgs& a, hipStream_t s);
// Fills its part of the arguments from the sizes and types.
void kv4_attention_plan(Kv4AttnArgs* a);
hipError_t launch_kv4_attention(const Kv4AttnArgs& a, hipStream_t s);
void launch_kv4_prompt(const Kv4AttnArgs& a, hipStream_t s);   // its part when a.rows >= 128

}  // namespace hr
