// Walk over (row, strip) tasks with a fixed stride: the strips of a row are
// consecutive tasks, one division at the start instead of one a task.
#pragma once

#include "device.cuh"

namespace avr {

struct StripWalk {
  int64_t row, row_step, task, task_step, tasks;
  int strip, strip_step, strips;
  __device__ __forceinline__ StripWalk(int64_t first, int64_t step, int64_t tasks_, int strips_)
      : task(first), task_step(step), tasks(tasks_), strips(strips_) {
    divide(first, row, strip);
    divide(step, row_step, strip_step);
  }
  __device__ __forceinline__ bool more() const { return task < tasks; }
  __device__ __forceinline__ void step() {
    task += task_step;
    row += row_step;
    strip += strip_step;
    if (strip >= strips) {
      strip -= strips;
      ++row;
    }
  }

 private:
  // the grid's warps are few: both dividends are below 2^32
  __device__ __forceinline__ void divide(int64_t x, int64_t& q, int& r) const {
    const uint32_t n = static_cast<uint32_t>(x), d = static_cast<uint32_t>(strips), k = n / d;
    q = k;
    r = static_cast<int>(n - k * d);
  }
};

}  // namespace avr
