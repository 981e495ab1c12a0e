/*
 * trellis_testing.h -- test and tuning hooks of libtrellis.so. Not part of
 * the layer's interface: production callers never need them.
 */
#ifndef TRELLIS_TESTING_H
#define TRELLIS_TESTING_H

#ifdef __cplusplus
extern "C" {
#endif

/* Decode table used by the prefill kernels of later calls, process-wide:
 *   -1  the library's own choice (the default),
 *    0  window -> float32 value table,
 *    1  window -> float16 code table,
 *    2  14-bit pair of windows -> two float16 codes (k = 2 only; other k keep
 *       the library's choice).
 * Every table gives the same weights; the hook lets tests run each table on
 * every k. Returns the previous setting, or -2 (and changes nothing) for a
 * value outside [-1, 2]. Thread-safe; a call already enqueued is not
 * affected. */
int trellis_test_force_table(int kind);

/* How later calls of the fine-tuned layers' entry points (trellis_adapters and
 * the ones declared after it) compute their product, process-wide:
 *   path   -1 the library's own choice (the default), 0 weights decoded in the
 *          product, 1 weights decoded once into the workspace;
 *   tiles  16-column tiles of weights decoded per launch with path 1, rounded
 *          up to whole workgroup tiles: 0 the library's own limit.
 * Both paths compute the same sums in different orders; the hook lets tests run
 * each on any number of rows, and several launches on a small matrix. Returns
 * 0, or -2 (and changes nothing) for a path outside [-1, 1] or tiles < 0.
 * Thread-safe; a call already enqueued is not affected. */
int trellis_test_force_path(int path, int tiles);

#ifdef __cplusplus
}
#endif

#endif /* TRELLIS_TESTING_H */
