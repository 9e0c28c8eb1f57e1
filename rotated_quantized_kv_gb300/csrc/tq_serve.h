// tq_serve.h -- private declarations of the serving calls (rotary positions,
// ragged writes and reads, tree attention): kernel parameters and launchers.
#pragma once

#include "tq_internal.h"

namespace tqk {

// ----------------------------------------------------------------- rotary positions
struct RopeTable {               // tq_rope_table
    double freq[TQ_MAX_HEAD_DIM / 2];
    double amplitude;
    int half, first, n;
    float *table;
};

struct RopeView {
    const float *table;          // [n_pos][2][half], or nullptr: no rotary positions
    int half, interleaved, n_pos;
};

struct RopeTensorParams {
    const void *in;
    void *out;
    int64_t is[3], os[3];        // strides of (b, h, t)
    int head0;                   // first head in the concatenation of the call's tensors
};

struct RopeParams {
    RopeView rope;
    const int *positions;
    int64_t pos_stride;
    int B, T, d, inverse;
    int n_tensors, heads;        // heads: over all tensors
    RopeTensorParams x[TQ_MAX_ROPE_TENSORS];
};
cudaError_t launch_rope_table(const RopeTable &p, cudaStream_t s);
cudaError_t launch_rope(const RopeParams &p, int dtype, cudaStream_t s);

// ----------------------------------------------------------------- segments
// A segment as the serving kernels address it: rows of (b, h, t).
struct SegView {
    int fp16;                    // fp16 segment: k, v are its rows
    int capacity;
    const uint8_t *k, *v;        // packed codes (or fp16 rows) of (0, 0, 0)
    const float *ks, *vs;        // packed: scales of (0, 0, 0)
    uint64_t kblock, vblock;     // bytes per batch element
    uint64_t koff[kMaxH], voff[kMaxH];  // byte offset of a head inside a batch block
    uint8_t kbits[kMaxH], vbits[kMaxH];
};

struct RowMap {                  // rows of a ragged write or read
    const int *t_begin, *n_rows; // n_rows: nullptr: n_max
    const int *slots;            // or (t_begin nullptr) the slot of row j in a pool of n_blocks pages
    int64_t slot_stride;
    int n_blocks;
    const int *index;            // source row of row j (writes), or nullptr
    int64_t index_stride;
    int n_max, n_source;
};

struct AppendParams {
    SegView seg;
    RowMap rows;
    RopeView rope;
    const int *positions;
    int64_t pos_stride;
    const uint16_t *K, *V;
    int64_t ks[3], vs[3];        // strides of (b, h, s)
    int B, H, d;
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d;
    float thr[kCbTotal];         // value thresholds, flat by bit width
    int law;
    uint32_t vwidths;            // bit b: some head's values have b bits
    int vec;                     // 8-byte loads of the source
};
cudaError_t launch_append(const AppendParams &p, cudaStream_t s);

// One thread per vector (head_dim 128), a launch per key and per value width: r.X,
// its strides and r.T (rows a sequence may get) describe the source rows.
struct AppendRowsParams {
    RowsParams r;
    RowMap rows;
    RopeView rope;               // keys
    const int *positions;
    int64_t pos_stride;
};
cudaError_t launch_append_keys(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_append_keys_slots(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_append_values(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_append_values_slots(const AppendRowsParams &p, int bits, bool beside, cudaStream_t s);

struct ReadParams {
    SegView seg;
    RowMap rows;
    void *K, *V;                 // either may be null
    int64_t ks[3], vs[3];
    int B, H, d;
    int rotate;                  // apply R
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d;
    float centroid[kCbTotal];
    uint32_t vwidths;            // bit b: some head's values have b bits
    int vec;                     // stores of four coordinates
};
cudaError_t launch_read(const ReadParams &p, int dtype, cudaStream_t s);

// One thread per vector of head_dim 128 or two of 64, a launch per key and per value width.
struct ReadRowsParams {
    RowMap rows;
    const uint8_t *codes;
    const float *scale;
    uint64_t block, off[kMaxH];
    int B, H, capacity, n_heads; // heads of this launch
    uint8_t head[kMaxH];
    void *out;
    int64_t st[3];
    int dtype, vec, rotate;      // vec: 16-byte stores
    uint32_t flip[32];           // record words: ones in the fields of the coordinates to negate
    float out_scale[kD];         // coordinates m and m + 64 of a thread's 128
    float level[256];            // values: the centroids
};
cudaError_t launch_read_keys(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_keys_slots(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_values(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_values_slots(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_keys_d64(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_keys_d64_slots(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_values_d64(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);
cudaError_t launch_read_values_d64_slots(const ReadRowsParams &p, int bits, bool beside, cudaStream_t s);

// ----------------------------------------------------------------- tree attention
// The work is a list of 128-token tiles.  For sequence b in order, KV head h,
// block of query rows rb (of R rows; row = draft * g + query head of the group):
// the tiles of b's packed segments, then those of its fp16 segments.  The workers
// take contiguous ranges of the list, all of the same length but the last.  The tiles of one (b, h, rb) are cut
// into parts: packed tiles every kTreePart, the fp16 ones likewise; every worker
// leaves one record (m, l, sum per row) for each part that it touches, at slot
// worker + part index (the pairs (worker, part) form a monotone path, so that
// the sums are distinct).  The merge adds the drafted tokens.
constexpr int kTreeTile = 128;
constexpr int kTreePart = 128;   // tiles: bounds the length of one tensor-core sum

struct TreeSeg {
    SegView seg;
    const int *len;              // per-sequence length or nullptr
    int n_tokens;
    int law;                     // value codebook
};

// What the merge needs of it: the list's geometry without the segments' data.
struct TreeListSeg {
    const int *len;
    int n_tokens;
};
struct TreeList {
    int B, H, g, N, R, n_rb;
    int n_seg, n_packed, ragged;
    int parts_packed, parts, workers;
    TreeListSeg seg[TQ_MAX_SEGMENTS];
};
struct TreeQueryParams {
    int H, g, n_rb, n_var, rows;  // rows: N g
    const uint16_t *q;
    int64_t qs[3];
    uint8_t *images;
    int *error;
    uint8_t var_bits[TQ_MAX_SEGMENTS][kMaxH];
    uint32_t sign_bits[4];       // (head_dim 64 and 128)
    float inv_sqrt_d, qk_scale;
};
struct TreeMergeParams {
    TreeList t;
    const uint16_t *q, *k, *v;
    int64_t qs[3], ks[3], vs[3];
    const uint32_t *mask;
    int64_t mask_stride;
    int mask_words;
    uint16_t *out;
    const float *part;
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d, qk_scale;
    int vec;                     // wide loads of q, k and v
};

struct TreeParams {
    int B, H, g, N, d, R, n_rb;  // g query heads per KV head, R rows per block, n_rb blocks
    int n_seg;                   // packed segments first
    int n_packed;
    int ragged;                  // some segment has per-sequence lengths
    int parts_packed, parts;     // parts per (b, h, rb): packed ones, all
    TreeSeg seg[TQ_MAX_SEGMENTS];
    const uint16_t *q, *k, *v;
    int64_t qs[3], ks[3], vs[3];
    const uint32_t *mask;
    int64_t mask_stride;
    int mask_words;
    uint16_t *out;
    float *part;                 // records: [slot][R][d + 4]: m (log2 units; any reference, the same for l and sum), l, pad, pad, sum
    // tensor-core form: the query blocks as MMA operands, one image per (b, h, rb) and
    // key width among the head's segments
    uint8_t *images;
    int n_var;
    uint8_t var[TQ_MAX_SEGMENTS][kMaxH];     // image of a segment
    uint8_t var_bits[TQ_MAX_SEGMENTS][kMaxH];  // key bits of image v (0: fp16 keys)
    int *error;
    int workers, wait_polls;
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d, qk_scale;  // qk_scale: log2(e) / sqrt(d)
    float centroid[2][kCbTotal]; // by law
};
// Rows per block, workers and the kernel's choice for a shape: the same rule
// sizes the workspace and launches the kernel.
struct TreeShape {
    int R, n_rb, workers;
};
// Value levels of the tensor-core form: fp16(s c_k) by law, flat by width, and 1/s.
struct TreeLevels {
    uint16_t half[2][kCbTotal];
    float inv[2][9];
};
// Whether a head dimension takes the tensor-core form (64 and 128).
inline bool tree_on_tensor_cores(int d) { return d == 64 || d == 128; }
cudaError_t launch_tree_mma(const TreeParams &p, cudaStream_t s);
// Bytes of a query image: hi and lo parts (rows of d fp16), 32 bytes a row for the
// constants' step, and the factor A.
inline size_t tree_image_bytes(int d, int R) { return (static_cast<size_t>(4) * d * R + 32 * R + 16 + 127) / 128 * 128; }
int tree_mma_rows(int rows);
// The levels of a value codebook as fp16(s c_k), s such that they round closely, and 1/s.
void value_levels(int law, int bits, const float *centroid, uint16_t *half, float *inv);
TreeShape tree_shape(int B, int H, int g, int N, int d, long long tiles_per_head);
cudaError_t launch_tree(const TreeParams &p, cudaStream_t s);

// ----------------------------------------------------------------- pages
struct PageParams {
    int B, page, width, n_pages;     // width: entries of a sequence's row of the table
    int n_max;
    int *table;
    int64_t table_stride;
    int *length;
    const int *count;                // tokens to place, or (release) to keep
    int *free_pages, *n_free;
    int *slots, *positions;          // [B][n_max], or nullptr
    int *granted;
};
cudaError_t launch_page_tables(const PageParams &p, cudaStream_t s);
cudaError_t launch_page_release(const PageParams &p, cudaStream_t s);

// ----------------------------------------------------------------- paged attention
// The (key bits, value bits) of a (segment, head) make its class (fp16 segments: 0, 0); the kernel
// of a class takes all that belong to it.  Its work is a list of stages of U tokens:
// sequence b in order, KV head h, block of R query heads rb, segment, stage.  The W workers
// take contiguous ranges of the list, equal to one stage (the first T, where there are
// fewer stages).  A worker leaves one record
// (m, l, sum per row) for each (b, h, rb) that it touches, at slot worker + (b H + h) n_rb +
// rb (along the list one or the other grows, so that the sums are distinct).
struct PagedSeg {
    SegView seg;                         // its batch elements are pages
    const int *table;                    // pages of a sequence, or nullptr: page b
    int64_t table_stride;
    int n_pages, page;                   // pages of the pool, tokens a page
    uint32_t magic;                      // t / page = t magic >> shift for 0 <= t < 2^31
    int shift;
};
struct PagedClass {
    int kb, vb, law;
    int R, n_rb;                         // query heads a block, and blocks of a KV head
    int n;                               // segments with heads of the class
    uint8_t seg[TQ_MAX_SEGMENTS];
    uint16_t heads[TQ_MAX_SEGMENTS];     // bit h: head h of that segment
    int unit, workers;                   // U, W
    int64_t part0;                       // first float of its records
};
constexpr int kPagedWarps = 12;          // workers an SM on the tensor cores
constexpr int kPagedClasses = 1 + TQ_MAX_SEGMENTS * kMaxH;
// What the list is made of: lengths without the segments' data.
struct PagedList {
    int B, H;
    const int *len[TQ_MAX_SEGMENTS];     // tokens of a sequence, or nullptr: limit
    int limit[TQ_MAX_SEGMENTS];          // most tokens a sequence can hold
};
struct PagedParams {
    PagedList list;
    PagedClass cls;                      // of this launch
    int g, d;
    PagedSeg seg[TQ_MAX_SEGMENTS];
    const uint16_t *q;
    int64_t qs[2];                       // strides of (b, head)
    float *part;                         // records, of a class [slot][R][d + 4]: m (log2 units), l, pad, pad, sum
    int *first;                          // [B + 1]: stages of the class before a sequence
    int first_class;                     // the call's first launch
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d, qk_scale;
    float centroid[kCbTotal];            // of the class's law
};
struct PagedMergeParams {
    PagedList list;
    int n_classes, g, d;
    uint16_t *out;                       // [B][H g][d]
    const float *part;
    const int *first;                    // [class][B + 1]
    int *error;
    PagedClass cls[kPagedClasses];
    uint32_t sign_bits[kMaxD / 32];
    float inv_sqrt_d;
};
// A class's stage length, rows a block and workers at once.
struct PagedShape {
    int unit, rows, workers;
};
PagedShape paged_shape(int d, bool packed);
cudaError_t launch_paged(const PagedParams &p, cudaStream_t s);
cudaError_t launch_paged_merge(const PagedMergeParams &p, cudaStream_t s);

// ----------------------------------------------------------------- verification of drafts
struct VerifyParams {
    int B, N, V;
    const int *tokens, *parents;         // parents nullptr: a chain
    int64_t tokens_stride, parents_stride;
    const void *target, *draft;          // draft nullptr: drafts without a distribution
    int64_t ts[2], ds[2];                // strides of (b, row)
    const float *uniform;
    int64_t uniform_stride;
    int *accepted, *n_accepted, *token;
};
cudaError_t launch_verify(const VerifyParams &p, int dtype, cudaStream_t s);

// ----------------------------------------------------------------- from tq_host.cpp
tq_status layout_status(const tq_segment_layout *L, bool need_bits);
void value_thresholds(float *flat, const uint8_t *bits, int H, int law);
void value_centroids(float *flat, const uint8_t *bits, int H, int law);
float rotation_scale(int d);
int decode_wait_polls();
int current_sm_count();
void fill_rows_rotation(RowsParams &p, const uint32_t *sign_bits, int d);
bool fill_rows_values(RowsParams &p, int bits, int law);

}  // namespace tqk
