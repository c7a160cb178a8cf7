// Shared by the host entry points (wfst_score_api.cpp) and the gfx950 kernels
// (wfst_layer.hip, wfst_norm.hip, wfst_sample.hip) of the operators around the
// search: the output layer with 4-bit weights, the log-softmax and the draw of
// tokens. Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

namespace wfst {

// Host helpers of wfst_api.cpp: record the calling thread's error message and
// return `code`; check a caller's device buffer (see there).
int api_fail(int code, const std::string &msg);
int api_check_buffer(const void *p, size_t bytes, int device, const char *what);

// Element types (the public WFST_LP_* values).
enum : int32_t { kF32 = 0, kF16 = 1, kBF16 = 2 };

inline size_t dtype_size(int32_t t) { return t == kF32 ? 4 : 2; }

// Rows of a padded [B, T] batch: row r = b * T + t holds data iff t < lengths[b]
// (every row when lengths is null). Rows without data are neither read nor written.
struct RowSet {
    const int32_t *lengths;
    int32_t T;
};

// ---- output layer

constexpr int kTileN = 16;      // output features of one weight tile
constexpr int kTileK = 128;     // input features of one weight tile

// A layer's device arrays. Weight tile (n / 16, k / 128) is 1024 bytes: 16 bytes
// for each of 64 lanes; lane l holds output feature l % 16, and its word j the
// features k = 32 j + 8 (l / 16) .. + 7 of the tile, feature 2p in bits 4p .. 4p+3
// and feature 2p + 1 in bits 16+4p .. 16+4p+3 (the order in which a shift and a
// mask yield the two halves of one register). Scales and zeros come gpt to a tile
// and feature, [n / 16][k / 128][n % 16][gpt]: 1 where groups are multiples of
// 128 features (a scale is repeated in each of its group's tiles), 2 for groups
// of 64, 4 (every 32 features) for all others.
struct Layer {
    const uint4 *w;
    const void *scales;         // binary32, or 16 bits as the caller gave them
    const uint8_t *zeros;       // null: 8
    const float *bias;          // null: 0
    int32_t K, N, group, gpt, kb, nt;
    int32_t scale_dtype;
};

struct LayerSource {
    const uint8_t *w;           // [N, ceil(K / 2)], feature 2i in the low half of byte i
    const void *scales;         // [N, ceil(K / group)]
    const uint8_t *zeros;       // the same shape, or null
    const float *bias;          // [N] or null
};

struct LayerCall {
    const void *x;
    void *out;
    int64_t x_stride, out_stride;
    int32_t M;
    int32_t x_dtype, out_dtype;
    RowSet rows;
    void *workspace;            // layer_workspace bytes
};

size_t layer_workspace(const Layer &l, int32_t rows, int32_t x_dtype);
hipError_t launch_layer_pack(const Layer &l, const LayerSource &src, uint4 *w, void *scales, uint8_t *zeros,
                             float *bias, hipStream_t s);
hipError_t launch_layer(const Layer &l, const LayerCall &c, hipStream_t s);

// ---- log-softmax

struct NormCall {
    const void *x;
    void *out;
    const float *bias;          // [V] or null
    int64_t x_stride, out_stride, rows;
    int32_t V;
    int32_t x_dtype, out_dtype;
    float scale;
    RowSet set;
    void *workspace;            // norm_workspace bytes
};

int norm_pieces(int32_t V, int32_t x_dtype, int32_t out_dtype);
size_t norm_workspace(int64_t rows, int32_t V, int32_t x_dtype, int32_t out_dtype);
hipError_t launch_log_softmax(const NormCall &c, hipStream_t s);

// ---- draw

struct SampleCall {
    const void *x;
    int64_t x_stride, rows;
    int32_t V, x_dtype;
    const float *u;
    float temperature, top_p, min_p;
    int32_t top_k;
    const float *temperatures, *top_ps, *min_ps;   // one a row, or null
    const int32_t *top_ks;
    int32_t *token;
    float *log_prob;            // may be null
    int32_t *kept;              // may be null
    RowSet set;
    void *workspace;            // sample_workspace bytes
};

int sample_chunks(int64_t rows, int32_t V, int32_t x_dtype);
size_t sample_workspace(int64_t rows, int32_t V, int32_t x_dtype);

hipError_t launch_sample(const SampleCall &c, hipStream_t s);

}  // namespace wfst
