// Arguments and launchers of a decode step's own kernels: block tables from
// lengths, the path through a drafted tree, the move of its slots, the rules on
// logits (internal to the library; the C ABI layer has validated everything here).
#pragma once

#include "kv_launch.h"

namespace q4 {

struct AssignArgs {
    const int32_t* table_in;
    int64_t table_in_stride;
    const int32_t* held_in;
    const int32_t* past;
    const int32_t* fresh;      // new tokens
    const int32_t* free_pages;
    const int32_t* free_count;
    const int32_t* parents;    // null: each token behind the one before it
    int32_t* table;
    int64_t table_stride;
    int32_t* held;
    int32_t* query_start;
    int32_t* context_len;
    int32_t* missing;
    int32_t* free_left;
    int32_t* positions;
    int64_t* slots;
    uint64_t* mask;            // null: none
    int mask_words, seqs, table_pages;
    FastDiv page;
    int64_t free_capacity, tokens;
    int per;                   // sequences of a workgroup
};
hipError_t launch_assign(AssignArgs a, hipStream_t s);

struct AcceptArgs {
    const int32_t* query_start;
    const int32_t* context_len;
    const int32_t* choice;
    const int32_t* draft;
    const int32_t* parents;    // null: a chain
    const int64_t* slots;      // null: every node has one
    int32_t* accepted;
    int32_t* next;
    int32_t* path;
    int32_t* lens;
    int32_t* history;          // null: none
    int64_t history_stride;
    int history_tokens, seqs;
    int64_t tokens;
};
hipError_t launch_accept(const AcceptArgs& a, hipStream_t s);

constexpr int kMoveLayers = 64;  // of one launch
struct MoveArgs {
    CacheArg cache;            // sizes and strides of every layer
    BatchArg batch;
    const int32_t* path;
    const int32_t* accepted;
    int64_t tokens;
    int layers;
    FastDiv units, chunks, heads;  // pieces of a sequence, of a head; kv heads
    char* at[2 * kMoveLayers];     // keys and values of each layer
};
hipError_t launch_move(MoveArgs& a, bool wide, hipStream_t s);

constexpr int kLogitKeys = 8;  // waves of a slice's workgroup
struct LogitArgs {
    const char* logits;
    int64_t row_stride, rows, vocab;
    float* out;                // null: none
    int64_t out_stride;
    int32_t* tokens;
    uint64_t* keys;            // [rows][slices][kLogitKeys], unless a slice is a row
    int64_t slices;
    int seqs;
    const int32_t* query_start;
    const int32_t* history;
    int64_t history_stride;
    int history_tokens;
    const int32_t* history_len;
    const int32_t* prompt_len;
    const int32_t* draft;
    const uint64_t* mask;
    int mask_words;
    const float* repetition;
    const float* presence;
    const float* frequency;
    const int32_t* bias_start;
    const int32_t* bias_tokens;
    const float* bias_values;
    int64_t biases;
    const uint32_t* allowed;
    int64_t allowed_stride, allowed_rows;
    const int32_t* allowed_row;
};
constexpr int64_t kLogitShort = 2048, kLogitLong = 8192;  // logits of a slice
constexpr int64_t kLogitFew = 512;                        // slices of a call for which one shorter than kLogitLong is taken
// Logits of one slice of a row: a rule on sizes, the same for the workspace and the launch.
int64_t logit_slice(int64_t rows, int64_t vocab);
hipError_t launch_logits(LogitArgs a, int type, hipStream_t s);

}  // namespace q4
